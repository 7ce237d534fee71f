// gemm_fp4.cu - the 4-bit block-scaled product on CTA pairs:
//   out[b, m, n] = bf16( g_x g_w sum_k (x sx)[b, m, k] (w sw)[b, n, k] + bias[n] )
// with E2M1 elements and one scale per 32 (MXFP4, E8M0) or 16 (NVFP4, E4M3)
// elements along K.  tcgen05.mma kind::mxf4 / kind::mxf4nvf4 with block scales,
// K = 64 per instruction, fp32 accumulation in tensor memory; the result is
// rounded once, after the tensor scales and the bias.
//
// A cluster of two CTAs computes one 256 x 256 output tile (or 256 x 128, see
// pair_plan) with cta_group::2: CTA r stages rows [128 r, +128) of the activation tile and of the weight tile,
// and receives the accumulator of its activation rows.  A stage is 128 bytes
// (256 elements) of K per row: four instructions, 512 cycles of the tensor
// cores.  One instruction reads the same bytes as an 8-bit one and does twice
// the work, and there are twice (MXFP4) or four times (NVFP4) as many scales
// per byte, which decides the rest:
//   scales: one TMA per operand brings a stage's atoms, and four warps write
//     them to tensor memory with tcgen05.st, a slot a stage, ahead of the MMAs.
//     (By tcgen05.cp between the MMAs, ~64 cycles an atom, M = 4096, N = 14336,
//     K = 4096 took 116 us instead of 89 in MXFP4's 6 atoms a stage and 145
//     instead of 94 in NVFP4's 12.  With fewer slots than stages the warps wait
//     for commits: half of NVFP4's atoms by cp, three slots, M = 8192, N = 4096, K
//     = 14336 139 us instead of 132.)
//   issue: the MMA warp stays converged and its instructions are predicated
//     (below): 89 -> 79 us.
//   tensor memory: the scale slots, and two accumulators of 256 columns that
//     overlap in what is left (from column ACC1 on).  The epilogue drains a tile's
//     shared columns first and releases them, so the next tile's MMAs run while
//     the rest is drained and stored.
// What bounds it (M = 4096, N = 14336, K = 4096, MXFP4 71.4 us, 6.7 PFLOP/s;
// NVFP4 77.3; tensor pipe busy 69 and 65 %): the way between L2 and the SMs,
// which operand loads (1.0 GB) and output stores share: without the stores 66
// of then 76 us, without the loads 68, without both 62; the tensor cores alone
// need 50.  Longer K writes less: M = 8192, N = 4096, K = 14336 124 us, 7.7
// PFLOP/s.  192-column tiles with two whole accumulators (86.8 against 73.1 us)
// load more.  Two pairs that share loads (a cluster of four; 144 of the 152 SMs
// hold them) have not been built, nor has the instruction with K = 96.
//
// Warps: 0 weight TMA, 1 tensor-memory allocation and (even CTA) MMA issue,
// 2 weight-scale TMA, 3 activation and activation-scale TMA, 4..7 scales into
// tensor memory, 8..15 epilogue.  Both CTAs' operand copies complete on the
// even CTA's `full` barrier; the MMA commits free a stage in both CTAs.
// Every wait is bounded; the cluster barriers are reached on every path.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_fp4.cuh"
#include "mx_kernels.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

namespace {

constexpr int BM = 128;       // activation rows per CTA (256 per pair)
constexpr int BKB = 128;      // bytes of K per row and stage
constexpr int BK = 2 * BKB;   // elements of K per stage
constexpr int MMA_K = 64;     // elements of K per instruction
constexpr int EPI_WARPS = 8;
constexpr int SF_WARPS = 4;
constexpr int THREADS = 128 + SF_WARPS * 32 + EPI_WARPS * 32;
constexpr int A_BYTES = BM * BKB;
constexpr int OUT_BOX = 32 * 128;  // staging box of an epilogue warp: 32 rows x 128 bytes, whole cache lines
constexpr int TMEM_COLS = 512;

// BN: output columns of a pair's tile, 256 or (few tiles) 128
template <int FMT, int BN>
struct Cfg {
  static constexpr int STAGES = BN == 256 ? 5 : (FMT == kQNV4 ? 6 : 7);
  static constexpr int NB = BN / 128;  // row tiles of the weights
  static constexpr int B_BYTES = (BN / 2) * BKB;
  // 512-byte atoms of 128 rows per stage: 128 (MXFP4) or 64 (NVFP4) elements each
  static constexpr int ATOMS = FMT == kQNV4 ? 4 : 2;
  static constexpr int SFA_BYTES = ATOMS * kAtomBytes;
  static constexpr int SFB_BYTES = ATOMS * NB * kAtomBytes;
  // Tensor memory: two accumulators, of 256 columns overlapping from column ACC1
  // on, then the scales: a slot a stage, ATOMS activation and NB ATOMS weight
  // atoms of 4 columns each.
  static constexpr int ACC1 = FMT == kQNV4 && BN == 256 ? 16 : 128;  // first column of the odd tiles' accumulator
  static constexpr int SLOT_COLS = ATOMS * 4 * (1 + NB);
  static constexpr int T_SF = ACC1 + BN;
  static_assert(T_SF + STAGES * SLOT_COLS <= TMEM_COLS, "tensor memory overflow");
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
  static constexpr int OFF_SFA = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_SFB = OFF_SFA + STAGES * SFA_BYTES;
  static constexpr int OFF_OUT = OFF_SFB + STAGES * SFB_BYTES;
  static constexpr int OFF_BIAS = OFF_OUT + EPI_WARPS * OUT_BOX;
  static constexpr int OFF_BAR = OFF_BIAS + EPI_WARPS * 4 * 32 * 2;
  static constexpr int OFF_MISC = OFF_BAR + (4 * STAGES + 2 + EPI_WARPS) * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 232448, "shared memory overflow");
};

// Instruction descriptor of kind::mxf4 / mxf4nvf4: E2M1 A and B (type code 1
// at bits 7 and 10), N >> 3 at bit 17, scale type at bit 23 (1 UE8M0, 0
// UE4M3), M >> 4 at bit 24; dense K = 64.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_fp4(uint32_t M, uint32_t N) {
  return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((FMT == kQMX4 ? 1u : 0u) << 23) | ((M >> 4) << 24);
}

// Issued by the lane whose `elected` is set, as a predicated instruction in code
// the whole warp runs: its operands then live in uniform registers (issued from
// a one-lane branch, each instruction costs ~115 cycles of moves, close to the
// 128 the tensor cores take for it).
template <int FMT>
__device__ __forceinline__ void mma_fp4_pair(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (FMT == kQMX4)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], "
        "p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void commit_pair_elected(uint32_t elected, uint64_t* bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(mask), "r"(elected)
      : "memory");
}

// TMA load by the elected lane; bar: shared-window address, either CTA of the pair.
__device__ __forceinline__ void tma_load_elected(uint32_t elected, uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                                 int c0, int c1, int c2) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
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

struct Args {
  const __nv_bfloat16* bias;
  const float* gx;
  const float* gw;
  int B, N;
  int MT, NT, KT;   // pair tiles, stages of K
  int last_steps;   // MMA steps of the last stage
  int units;        // tiles * splits
  int splits;
  int exchange;     // 1: the two splits of a tile meet in a cluster of two pairs
  int n_fast;       // tile order: 1 = column tiles vary fastest
};

// Unit u = tile * splits + s: its tile and stages [kt_lo, kt_hi).
__device__ __forceinline__ void unit_coords(int u, const Args& a, int& b, int& mt, int& nt, int& s, int& kt_lo,
                                            int& kt_hi) {
  const int tile = u / a.splits;
  s = u - tile * a.splits;
  const int per_b = a.MT * a.NT;
  b = tile / per_b;
  const int t = tile - b * per_b;
  if (a.n_fast) {
    mt = t / a.NT;
    nt = t - mt * a.NT;
  } else {
    nt = t / a.MT;
    mt = t - nt * a.MT;
  }
  kt_lo = s * a.KT / a.splits;
  kt_hi = (s + 1) * a.KT / a.splits;
}

template <int FMT, int BN>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSFA, const __grid_constant__ CUtensorMap tmSFB,
                    const __grid_constant__ CUtensorMap tmOut, const Args args) {
  using C = Cfg<FMT, BN>;
  constexpr int STAGES = C::STAGES, B_BYTES = C::B_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* sf_full = empty + STAGES;
  uint64_t* sf_ready = sf_full + STAGES;
  uint64_t* acc_full = sf_ready + STAGES;
  uint64_t* acc_free = acc_full + 1;
  uint64_t* received = acc_free + 1;  // [EPI_WARPS]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  // clusters are (2, 1, 1), or (4, 1, 1) with the two K splits of a tile
  const uint32_t crank = cluster_ctarank() & 3u;
  const uint32_t rank = crank & 1u, even = crank & 2u;
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;

  if (warp == 0) {
    // full, empty, sf_full: one arrival (the even CTA's copy of full is used, and
    // empty is the even CTA's commit); sf_ready: both CTAs' scale writers
    if (lane < 4 * STAGES) mbar_init(&full[lane], lane < 3 * STAGES ? 1 : 2 * SF_WARPS);
    if (lane < EPI_WARPS) mbar_init(&received[lane], 1);
    if (lane == 0) {
      mbar_init(acc_full, 1);
      mbar_init(acc_free, 2 * EPI_WARPS);
      *abort_flag = 0;
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 64) {
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmSFB);
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmSFA);
    prefetch_tmap(&tmOut);
  }
  __syncthreads();
  cluster_arrive_relaxed();
  cluster_wait();  // both CTAs' barriers exist before anyone signals them
  // This call's reduce waits for this grid itself.  Without a split the next
  // kernel is not let in early: a quantise or activation kernel that starts
  // beside this one keeps its shared-memory split of the SM, and with the L1
  // that is left a 8192 x 14336 quantise took 59 us instead of 46.
  if (args.splits > 1 && !args.exchange && threadIdx.x == 0) launch_dependents();
  uint32_t tmem = 0;
  if (warp == 1 || warp >= 4) {
    // the loads start without waiting for the allocation
    if (warp == 1) {
      tmem_alloc_pair(tmem_slot, TMEM_COLS);
      tmem_relinquish_pair();
    }
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS - 96) : "memory");
    tc_fence_after();
    tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  }

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------ producers
    // Warp 0 the weights, 2 their scales, 3 the activations and theirs (after
    // the kernel before this one in the stream, whose output they are).
    // Operands of both CTAs complete on the even CTA's `full`, whose count the
    // even CTA alone posts, the scales on this CTA's own sf_full.  Bytes may
    // land before the count is posted, but not a phase early: the stage was
    // freed by a commit behind the MMA that waited for the previous phase.
    const uint32_t elected = elect_one();
    const uint32_t poster = leader ? elected : 0u;
    const uint32_t base = smem_u32(smem);
    const uint32_t full_even = map_shared_rank(smem_u32(full), even), sf_own = map_shared_rank(smem_u32(sf_full), crank);
    if (warp == 3) grid_dependency_wait();
    int stage = 0;
    uint32_t phase = 1;  // the first round's slots are free
    int64_t issued = 0;
    bool ok = true;
    for (int u = pair; ok && u < args.units; u += npairs) {
      int b, mt, nt, sp, kt, kt_hi;
      unit_coords(u, args, b, mt, nt, sp, kt, kt_hi);
      const int rt = mt * 2 + static_cast<int>(rank);
      for (; kt < kt_hi; ++kt, ++issued) {
        if (!mbar_wait_warp(&empty[stage], phase, abort_flag)) {
          ok = false;
          break;
        }
        if (warp == 0) {
          expect_tx_elected(poster, smem_u32(&full[stage]), 2 * (A_BYTES + B_BYTES));
          tma_load_elected(elected, base + C::OFF_B + stage * B_BYTES, &tmB, full_even + stage * 8, kt * BKB,
                           nt * BN + static_cast<int>(rank) * (BN / 2), b);
        } else if (warp == 2) {
          expect_tx_elected(elected, smem_u32(&sf_full[stage]), C::SFA_BYTES + C::SFB_BYTES);
          tma_load_elected(elected, base + C::OFF_SFB + stage * C::SFB_BYTES, &tmSFB, sf_own + stage * 8,
                           nt * C::NB * (kAtomBytes / 4), kt * C::ATOMS, b);
        } else {
          tma_load_elected(elected, base + C::OFF_A + stage * A_BYTES, &tmA, full_even + stage * 8, kt * BKB, rt * BM,
                           b);
          tma_load_elected(elected, base + C::OFF_SFA + stage * C::SFA_BYTES, &tmSFA, sf_own + stage * 8,
                           rt * (kAtomBytes / 4), kt * C::ATOMS, b);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // Before exit: every commit to this CTA's empty barriers has arrived; a
    // stage's last commit follows the MMA that waited for its copies.
    if (lane == 0) {
      for (int s = 0; s < STAGES; ++s) {
        if (issued <= s) continue;
        const int64_t last = ((issued - 1 - s) / STAGES) * STAGES + s;
        mbar_wait(&empty[s], static_cast<uint32_t>((last / STAGES) & 1), nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader) {
      constexpr uint32_t idesc = idesc_fp4<FMT>(2 * BM, BN);
      const uint32_t elected = elect_one();
      const uint16_t pair_mask = static_cast<uint16_t>(0x3u << even);
      const uint64_t ad0 = sdesc_kmajor_sw128(smem_u32(smem + C::OFF_A));
      const uint64_t bd0 = sdesc_kmajor_sw128(smem_u32(smem + C::OFF_B));
      int stage = 0, tile_no = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < args.units; u += npairs, ++tile_no) {
        const int sp = u % args.splits;
        const int kt_lo = sp * args.KT / args.splits, kt_hi = (sp + 1) * args.KT / args.splits;
        const uint32_t acc = tmem + ((tile_no & 1) ? C::ACC1 : 0);
        // the columns shared with the previous tile's accumulator are drained
        if (tile_no > 0 && !mbar_wait_warp(acc_free, static_cast<uint32_t>((tile_no - 1) & 1), abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kt = kt_lo; kt < kt_hi; ++kt) {
          // operands landed (the even CTA's scale writers waited for them) and
          // both CTAs' scales in tensor memory
          if (!mbar_wait_warp(&sf_ready[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = ad0 + static_cast<uint32_t>(stage * (A_BYTES >> 4));
          const uint64_t bd = bd0 + static_cast<uint32_t>(stage * (B_BYTES >> 4));
          const int steps = kt == args.KT - 1 ? args.last_steps : BK / MMA_K;
          const uint32_t t_sfa = tmem + C::T_SF + stage * C::SLOT_COLS;
          const uint32_t t_sfb = t_sfa + 4 * C::ATOMS;
#pragma unroll
          for (int kk = 0; kk < BK / MMA_K; ++kk) {
            // MXFP4: two steps share an atom (scale bytes 0-1 and 2-3)
            const int j = FMT == kQNV4 ? kk : kk >> 1;
            const uint32_t id = FMT == kQNV4 ? 0u : static_cast<uint32_t>(kk & 1) * 2u;
            mma_fp4_pair<FMT>(kk < steps ? elected : 0u, acc, ad + 2 * kk, bd + 2 * kk,
                              idesc_with_sf_id(idesc, id, id), t_sfa + 4 * j, t_sfb + 4 * C::NB * j,
                              ((kt - kt_lo) | kk) != 0);
          }
          commit_pair_elected(elected, &empty[stage], pair_mask);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit_pair_elected(elected, acc_full, pair_mask);
      }
      // Before exit: the last signals that the accumulators are drained, which the odd
      // CTA sends here.  (Ordered by a releasing barrier at the end instead, N = 14336, K
      // = 4096, M = 128 took 10.0 us, not 9.2; N = K = 4096, M = 512 8.95, not 8.7.)
      if (ok && !args.exchange && tile_no > 0)
        ok = mbar_wait_warp(acc_free, static_cast<uint32_t>((tile_no - 1) & 1), abort_flag);
      if (!ok) __nanosleep(200000);  // let issued tensor-core work retire
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + SF_WARPS) {
    // ------------------------------------------------------------ scale writers
    // Each warp writes its 32 lanes of every atom: line l of an atom (rows l,
    // l + 32, l + 64, l + 96) goes to lane l of each quarter.
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::T_SF;
    const uint32_t ready_even = map_shared_rank(smem_u32(sf_ready), even);
    int64_t total = 0;
    for (int u = pair; u < args.units; u += npairs) {
      const int sp = u % args.splits;
      total += (sp + 1) * args.KT / args.splits - sp * args.KT / args.splits;
    }
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t i = 0; i < total; ++i) {
      // the stage's slot is free: its refill has waited for the MMAs that read it
      if (!mbar_wait(&sf_full[stage], phase, abort_flag)) break;
      tc_fence_after();
      const uint4* sa = reinterpret_cast<const uint4*>(smem + C::OFF_SFA + stage * C::SFA_BYTES) + lane;
      const uint4* sb = reinterpret_cast<const uint4*>(smem + C::OFF_SFB + stage * C::SFB_BYTES) + lane;
      const uint32_t t = lane_base + stage * C::SLOT_COLS;
#pragma unroll
      for (int j = 0; j < C::ATOMS; ++j) {
        const uint4 v = sa[j * 32];
        tmem_st_32x32b_x4(t + 4 * j, v.x, v.y, v.z, v.w);
      }
#pragma unroll
      for (int j = 0; j < C::NB * C::ATOMS; ++j) {
        const uint4 v = sb[j * 32];
        tmem_st_32x32b_x4(t + 4 * C::ATOMS + 4 * j, v.x, v.y, v.z, v.w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (!leader)
          mbar_arrive_remote(ready_even + static_cast<uint32_t>(stage * 8));
        else if (mbar_wait(&full[stage], phase, abort_flag))
          mbar_arrive(&sf_ready[stage]);
      }
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp >= 4 + SF_WARPS) {
    // ------------------------------------------------------------ epilogue
    // Warp e drains lanes 32 (warp % 4).. of the tile's group e / 4 of 64 columns
    // and, of 256 columns, the one two further.  The group that shares columns
    // with the next tile's accumulator comes first (the upper one of an even
    // tile, the lower one of an odd one), and the shared columns are released
    // once all of them are in registers, before anything is stored.
    const int ew = warp - 4 - SF_WARPS;
    const int quad = warp & 3;
    const int half = ew >> 2;
    uint8_t* box = smem + C::OFF_OUT + ew * OUT_BOX;
    __nv_bfloat16* bias_s = reinterpret_cast<__nv_bfloat16*>(smem + C::OFF_BIAS) + ew * 128;
    const uint32_t acc_free_even = map_shared_rank(smem_u32(acc_free), even);
    grid_dependency_wait();  // g_x may be the previous kernel's output
    float alpha = 1.f;
    if (args.gx != nullptr) alpha = *args.gx;
    if (args.gw != nullptr) alpha *= *args.gw;
    const bool partial = args.splits > 1 && !args.exchange;
    bool pending = false;
    // 16-byte piece q of this lane's row: 128-byte swizzle, so the eight lanes
    // of a store phase touch different banks
    auto piece = [&](int q) { return reinterpret_cast<uint4*>(box + lane * 128 + ((q ^ (lane & 7)) << 4)); };
    auto box_free = [&]() {
      if (lane == 0 && pending) bulk_wait_group_read0();
      __syncwarp();
    };
    auto store_box = [&](int col, int row, int z) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&tmOut, box, col, row, z);
        bulk_commit_group();
        pending = true;
      }
    };
    // bias and rounding of a 64-column group of this lane's row, and its store
    auto finish = [&](const uint32_t (&r)[2][32], const __nv_bfloat16* bias_g, int col, int row, int z) {
      const uint32_t* bw = reinterpret_cast<const uint32_t*>(bias_g);
      box_free();
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 4 * q + e;  // columns 2 j and 2 j + 1 of the group
          float lo = __uint_as_float(r[j >> 4][2 * (j & 15)]), hi = __uint_as_float(r[j >> 4][2 * (j & 15) + 1]);
          if (args.bias != nullptr) {
            lo = fmaf(lo, alpha, __uint_as_float(bw[j] << 16));
            hi = fmaf(hi, alpha, __uint_as_float(bw[j] & 0xFFFF0000u));
          } else {
            lo *= alpha;
            hi *= alpha;
          }
          o[e] = pack_bf16x2(lo, hi);
        }
        *piece(q) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      store_box(col, row, z);
    };
    if (BN == 256 && args.exchange) {
      // The pair's sum over its half of K; each of the two pairs of the cluster
      // finishes half of the columns and sends the other half, in fp32, to the
      // other pair: staged where its own weight stages were (every copy and MMA
      // of this pair is done once the accumulator is), copied to where the other
      // pair's activation stages were (free after the cluster barrier).  Warp e
      // sends what warp e of the other CTA reads: 32 rows of one group, 16-byte
      // piece q of lane l at 512 q + 16 l.
      int b, mt, nt, sp, kt_lo, kt_hi;
      unit_coords(pair, args, b, mt, nt, sp, kt_lo, kt_hi);
      const int row0 = (mt * 2 + static_cast<int>(rank)) * BM + quad * 32;
      const int keep = (2 * sp + half) * 64, send = (2 * (1 - sp) + half) * 64;
      if (args.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = nt * BN + keep + i * 32 + lane;
          bias_s[i * 32 + lane] = n < args.N ? args.bias[n] : __float2bfloat16(0.f);
        }
      }
      const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full, 0, abort_flag));
      cluster_arrive_relaxed();
      const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      uint32_t r[2][32];
      uint8_t* out_box = smem + C::OFF_B + ew * 8192;
      uint8_t* in_box = smem + C::OFF_A + ew * 8192;
      tc_fence_after();
      if (got) {
        tmem_ld_32x32b_x32(acc + send, r[0]);
        tmem_ld_32x32b_x32(acc + send + 32, r[1]);
        tmem_ld_wait();
        uint4* o = reinterpret_cast<uint4*>(out_box) + lane;
#pragma unroll
        for (int q = 0; q < 16; ++q)
          o[q * 32] = make_uint4(r[q >> 3][4 * (q & 7)], r[q >> 3][4 * (q & 7) + 1], r[q >> 3][4 * (q & 7) + 2],
                                 r[q >> 3][4 * (q & 7) + 3]);
        fence_proxy_async_smem();
        __syncwarp();
      }
      cluster_wait();
      if (lane == 0) {
        mbar_arrive_expect_tx(&received[ew], 8192);
        if (got)
          bulk_copy_cluster(map_shared_rank(smem_u32(in_box), crank ^ 2u), out_box, 8192,
                            map_shared_rank(smem_u32(&received[ew]), crank ^ 2u));
      }
      if (got) {
        tmem_ld_32x32b_x32(acc + keep, r[0]);
        tmem_ld_32x32b_x32(acc + keep + 32, r[1]);
        tmem_ld_wait();
      }
      __syncwarp();
      // waited for even without a sum of our own: no copy may land after we leave
      const bool came = __all_sync(0xFFFFFFFFu, mbar_wait(&received[ew], 0, nullptr));
      if (got && came) {
        const uint4* in = reinterpret_cast<const uint4*>(in_box) + lane;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint4 v = in[q * 32];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t& x = r[q >> 3][4 * (q & 7) + e];
            x = __float_as_uint(__uint_as_float(x) + __uint_as_float(w[e]));
          }
        }
        finish(r, bias_s, nt * BN + keep, row0, b);
      }
    } else {
      int tile_no = 0;
      for (int u = pair; u < args.units; u += npairs, ++tile_no) {
        int b, mt, nt, sp, kt_lo, kt_hi;
        unit_coords(u, args, b, mt, nt, sp, kt_lo, kt_hi);
        const int row0 = (mt * 2 + static_cast<int>(rank)) * BM + quad * 32;
        if (!partial && args.bias != nullptr) {
          // the bias of this warp's two groups (zero past N)
#pragma unroll
          for (int i = 0; i < 2 * C::NB; ++i) {
            const int n = nt * BN + (half + (i & 2)) * 64 + (i & 1) * 32 + lane;
            bias_s[i * 32 + lane] = n < args.N ? args.bias[n] : __float2bfloat16(0.f);
          }
          __syncwarp();
        }
        if (!mbar_wait(acc_full, static_cast<uint32_t>(tile_no & 1), abort_flag)) break;
        tc_fence_after();
        const bool odd = tile_no & 1;
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (odd ? C::ACC1 : 0);
        // whether the second groups hold shared columns too
        constexpr int kReleased = C::ACC1 < 64 ? 1 : 0;
#pragma unroll 1
        for (int i = 0; i < C::NB; ++i) {
          const int up = C::NB == 2 && (i == 0) != odd;  // the upper of this warp's groups
          const int col = (half + 2 * up) * 64;
          uint32_t r[2][32];
          tmem_ld_32x32b_x32(acc + col, r[0]);
          tmem_ld_32x32b_x32(acc + col + 32, r[1]);
          tmem_ld_wait();
          if (i == kReleased) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(acc_free_even);
          }
          if (C::NB == 2 && i == 1 && !partial && u + npairs >= args.units) {
            // the last tile: its second group goes where activation stages were,
            // without waiting for the first box to be read
            box = smem + C::OFF_A + ew * OUT_BOX;
            pending = false;
          }
          if (partial) {
            // fp32 partial of this K split: 32 columns a box
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              box_free();
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *piece(q) = make_uint4(__float_as_uint(__uint_as_float(r[h][4 * q]) * alpha),
                                       __float_as_uint(__uint_as_float(r[h][4 * q + 1]) * alpha),
                                       __float_as_uint(__uint_as_float(r[h][4 * q + 2]) * alpha),
                                       __float_as_uint(__uint_as_float(r[h][4 * q + 3]) * alpha));
              store_box(nt * BN + col + 32 * h, row0, sp * args.B + b);
            }
            continue;
          }
          finish(r, bias_s + up * 64, nt * BN + col, row0, b);
        }
      }
    }
    if (lane == 0) bulk_wait_group_read0();  // the boxes are read; the end of the grid completes the stores
    __syncwarp();
  }

  tc_fence_before();
  __syncwarp();
  if (BN == 256 && args.exchange && warp < 4 + SF_WARPS) {  // the epilogue's barrier
    cluster_arrive_relaxed();
    cluster_wait();
  }
  cluster_arrive_last(*abort_flag);
  cluster_wait();  // no CTA of the cluster leaves while another may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

struct PairPlan {
  int bn, splits;
  bool exchange;  // the two splits meet in a cluster, without partials in memory
  int64_t cost;
};

template <int FMT, int BN>
cudaError_t launch_t(const Fp4Problem& p, const PairPlan& plan, int sms, cudaStream_t stream, const char** msg) {
  using C = Cfg<FMT, BN>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(gemm_fp4_kernel<FMT, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) {
      *msg = "cudaFuncSetAttribute(max dynamic shared memory) failed";
      return e;
    }
    attr_set[dev] = true;
  }
  const bool exchange = plan.exchange;
  const int splits = plan.splits;
  const bool partials = splits > 1 && !exchange;
  const int64_t RTA = ceil_div(p.M, kAtomRows), RTB = ceil_div(p.N, kAtomRows);
  const int64_t KA = ceil_div(fp4_scale_extent(FMT, p.K), kTileK);  // scale atoms along K
  const int64_t kb = p.K / 2;
  CUtensorMap ma, mb, msa, msb, mo;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const int words = kAtomBytes / 4;
  bool ok = encode_map3(&ma, u8, p.x, kb, p.M, p.B, kb, p.M * kb, BKB, BM, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B) &&
            encode_map3(&mb, u8, p.w, kb, p.N, p.B, kb, p.N * kb, BKB, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B) &&
            encode_map3(&msa, u32, p.sfx, RTA * words, KA, p.B, RTA * kAtomBytes, KA * RTA * kAtomBytes, words, C::ATOMS,
                    CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) &&
            encode_map3(&msb, u32, p.sfw, RTB * words, KA, p.B, RTB * kAtomBytes, KA * RTB * kAtomBytes, C::NB * words,
                    C::ATOMS, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (partials)
    ok = ok && encode_map3(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.part, p.N, p.M, splits * p.B, p.N * 4, p.M * p.N * 4, 32,
                       32, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
  else
    ok = ok && encode_map3(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.out, p.N, p.M, p.B, p.N * 2, p.M * p.N * 2, 64, 32,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
  if (!ok) {
    *msg = "cuTensorMapEncodeTiled rejected a 4-bit operand or output";
    return cudaErrorInvalidValue;
  }
  Args a;
  a.bias = partials ? nullptr : static_cast<const __nv_bfloat16*>(p.bias);
  a.gx = p.gx;
  a.gw = p.gw;
  a.B = static_cast<int>(p.B);
  a.N = static_cast<int>(p.N);
  a.MT = static_cast<int>(ceil_div(p.M, 2 * BM));
  a.NT = static_cast<int>(ceil_div(p.N, BN));
  a.KT = static_cast<int>(ceil_div(p.K, BK));
  a.last_steps = static_cast<int>(ceil_div(p.K - static_cast<int64_t>(a.KT - 1) * BK, MMA_K));
  a.splits = splits;
  a.exchange = exchange ? 1 : 0;
  a.units = a.B * a.MT * a.NT * splits;
  // Column tiles fastest while a sweep of the weights stays in L2 (two dies:
  // half of it) or they are the operand with fewer bytes: M = 4096, N = 14336, K =
  // 4096 75.0 -> 71.4 us, M = 8192, N = 4096, K = 14336 132.4 -> 126.8 us; at N =
  // 28672, K = 4096 (59 MB of weights) row tiles fastest 144.1 against 155.9.  Up
  // to eight row tiles the first wave would take in all of the weights: row tiles
  // fastest, weights from HBM, N = 14336, K = 4096, M = 1024 22.5 -> 21.6, M = 2048
  // 40.8 -> 39.7 us (in L2 20.3 and 38.4 -> 39.4).
  a.n_fast = a.MT > 8 && (p.M >= p.N || p.N * p.K / 2 <= (32ll << 20)) ? 1 : 0;
  const int pairs = exchange || a.units < sms / 2 ? a.units : sms / 2;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = exchange ? 4 : 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_fp4_kernel<FMT, BN>, ma, mb, msa, msb, mo, a);
  if (e != cudaSuccess) {
    *msg = "4-bit GEMM launch failed";
    return e;
  }
  if (partials) {
    e = launch_splitk_reduce(p.part, splits, p.B, p.M, p.N, p.bias, p.out, nullptr, nullptr, sms, stream);
    if (e != cudaSuccess) *msg = "split-K reduce launch failed";
  }
  return e;
}

}  // namespace

bool encode_map3(CUtensorMap* m, CUtensorMapDataType dtype, const void* base, int64_t d0, int64_t d1, int64_t d2,
             int64_t s1, int64_t s2, int b0, int b1, CUtensorMapSwizzle sw, CUtensorMapL2promotion l2) {
  EncodeTiledFn encode = encode_tiled_fn();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1), static_cast<cuuint64_t>(s2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(b0), static_cast<cuuint32_t>(b1), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(m, dtype, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, l2,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// How a product runs on CTA pairs (a function of the shape alone) and what it
// costs, in 0.01 us: the least of
//   256-column tiles: 4.6 us + 0.26 us a stage of K (0.36 where a row of K/2
//     bytes is not a whole number of 128-byte lines);
//   128-column tiles, where one a pair covers the output: 4.15 us + 0.25 (0.28)
//     us a stage.  A CTA still loads 24 of the 32 KB a stage, so only the
//     epilogue and the misaligned loads get shorter;
//   256-column tiles with K split in two, the halves meeting in a cluster of two
//     pairs: 1.3 us + 0.04 us a tile more;
//   256-column tiles with K split over about 64 pairs, at least four stages
//     each: partial sums and the kernel that adds them cost 2.9 us + 0.18 us a
//     tile more.
// Measured (us, MXFP4, 256 / 128 columns / in two / split): N = K = 4096, M = 512
// 9.0 / 8.5 / 8.7 / 15.0, M = 768 (one tile a pair / two) 9.8 / 13.5; N = K =
// 2048, M = 512 6.7 / 6.2 / 7.1 / 10.4; N = K = 8192, M = 256 13.4 / 12.5 / 11.3 /
// 17.5; N = 1000, K = 4128, M = 768 11.0 / 8.9 / 9.4 / 11.2; N = 4096, K = 14336,
// M = 256 19.5 / 18.4 / 13.5 / 13.9, M = 512 19.5 / 18.7 / 14.5 / 20.9; N = 1024,
// K = 28672, M = 512 34.1 / 32.5 / 20.9 / 13.2.
PairPlan pair_plan(int64_t B, int64_t M, int64_t N, int64_t K, bool may_split) {
  const int64_t stages = ceil_div(K, BK), rows = B * ceil_div(M, 2 * BM), tiles = rows * ceil_div(N, 256);
  const bool lines = K % BK == 0;
  const int64_t stage = lines ? 26 : 36;
  PairPlan p = {256, 1, false, 460 + stage * stages * (tiles > 76 ? ceil_div(tiles, 76) : 1)};
  const int64_t narrow = 415 + (lines ? 25 : 28) * stages;
  if (rows * ceil_div(N, 128) <= 76 && narrow < p.cost) p = {128, 1, false, narrow};
  // 36 clusters of four CTAs run at a time
  const int64_t exchange = 460 + stage * ceil_div(stages, 2) + 130 + 4 * tiles;
  if (tiles <= 36 && stages >= 2 && exchange < p.cost) p = {256, 2, true, exchange};
  int64_t s = tiles > 0 ? 64 / tiles : 1;
  if (s > stages / 4) s = stages / 4;
  if (s > 8) s = 8;
  if (!may_split || s < 2) return p;
  const int64_t split = 460 + stage * ceil_div(stages, s) + 290 + 18 * tiles;
  if (split < p.cost) p = {256, static_cast<int>(s), false, split};
  return p;
}

}  // namespace

int fp4_splitk_splits(int64_t B, int64_t M, int64_t N, int64_t K) {
  const PairPlan p = pair_plan(B, M, N, K, true);
  return p.exchange ? 1 : p.splits;
}

int64_t fp4_pair_cost(int64_t B, int64_t M, int64_t N, int64_t K) { return pair_plan(B, M, N, K, true).cost; }

cudaError_t launch_gemm_fp4(const Fp4Problem& p, int sms, cudaStream_t stream, const char** msg) {
  const PairPlan plan = pair_plan(p.B, p.M, p.N, p.K, p.part != nullptr && p.splits > 1);
  if (plan.bn == 128)
    return p.fmt == kQNV4 ? launch_t<kQNV4, 128>(p, plan, sms, stream, msg)
                          : launch_t<kQMX4, 128>(p, plan, sms, stream, msg);
  return p.fmt == kQNV4 ? launch_t<kQNV4, 256>(p, plan, sms, stream, msg)
                        : launch_t<kQMX4, 256>(p, plan, sms, stream, msg);
}

cudaError_t take_status_fp4(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
}

}  // namespace mx
