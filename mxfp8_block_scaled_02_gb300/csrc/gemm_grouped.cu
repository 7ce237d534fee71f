// gemm_grouped.cu - products grouped by expert, and the block-128 FP8 product:
//   out[r, n] = bf16( sum_k x[r, k] w[e(r), n, k] + bias[e(r), n] )
// for rows r sorted by group: group e owns rows [offsets[e], offsets[e + 1]).  A
// dense or batched product is the case of groups of equal length (offsets null).
// Elements are E4M3; the scales are either
//   MXFP8    one E8M0 scale per 32 elements along K of x and of w: applied by the
//            tensor cores (kind::mxf8f6f4.block_scale), sums stay in tensor memory;
//   fp8_128  one fp32 scale per 128 elements of x along K, one per 128 x 128 block
//            of w: kind::f8f6f4 makes the sum of one block of K, and the epilogue
//            warps add it to their fp32 registers times s_x s_w.
//
// The weights are the MMA's M side (128 rows a CTA) and the rows of x its N side,
// because the groups are ragged in x: a tile takes as many columns as its group
// has rows left, in steps of 16 (32 on a pair), and a group's rows are shared out
// evenly over its tiles, so hardly any MMA column is padding.  Two shapes:
//   CG = 2: 256 weight rows x up to 256 rows of x on a pair of CTAs (cta_group::2;
//           MXFP8, fp8_128 has gemm_b128_pair.cu), where the way between L2 and the
//           SMs bounds the product: 64 KB a stage and pair;
//   CG = 1: 128 weight rows x up to 16, 32, 64 or 128 on one CTA, where reading
//           the weights does.  With few tiles K is split over a cluster of S CTAs,
//           whose partial sums meet in distributed shared memory (TN <= 64).
// CTAs are persistent and find their tiles from the offsets, which are read on
// the device: nothing about the groups is known to the host.
//
// Accumulators have weight rows in lanes and rows of x in columns, the transpose
// of the output.  The epilogue reads them as 16 x 256-bit fragments, in which a
// thread holds two neighbouring columns of four lanes: a warp then needs each
// column's fp8_128 scale once per 16-byte shared-memory read of 16 columns (with a
// lane per row every thread would read all of them), and stmatrix.trans turns the
// fragments of bf16 into rows of the output.
//
// Measured (us, weights from HBM, in a CUDA graph, x quantised before): MXFP8, 128
// rows on 54 of 64 experts of 2048 x 4096 73 (6.4 TB/s of weights); 16384 rows on 13
// of 16 experts of 4096 x 4096 185 with the repack of x's scale words (2.97 PFLOP/s;
// 205 before the MMA warp waited for the operands itself and a second set of scale
// warps took every other stage, 167 without the scales' tensor-memory stores).
// fp8_128: eight rows on eight experts of 2048 x 4096 15.7 (4.3 TB/s: 128 tiles on 152
// SMs, and ~4 us of chain); one row, N = K = 4096, bf16 x quantised inside 7.8 (8.6 with
// a warp a stage, which loaded x cold and met the instruction cache's misses after the
// kernel before had ended), of which two thirds are the chain from launch to the
// exchange.
//
// Warps: 0 weight TMA (and, MXFP8, weight scales), 1 tensor-memory allocation and
// MMA issue, 2 TMA of x, 3 the group table and the scales of fp8_128; MXFP8: 4..7
// (on pairs the last four too) scales into tensor memory; the epilogue, 4 or 8
// warps; with kQuant four that quantise x.  Every wait is bounded and the cluster
// barriers are reached on every path.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_block128.cuh"
#include "mx_grouped.cuh"
#include "mx_kernels.h"
#include "mx_layout.cuh"
#include "mx_ptx.cuh"

namespace mx {

namespace {

constexpr int ROWS = kGW_Rows, BK = kGBK, BOX = kGBox;
constexpr int W_BYTES = ROWS * BK;
using Args = GroupedArgs;
using Tile = GroupTile;

// K splits: what a CTA of a cluster of S receives, 4 KB of each CTA for each group of 8
// columns that it finishes, and the room for it.
constexpr int received_bytes(int tn, int splits) { return (tn / 8 + splits - 1) / splits * splits * 4096; }
constexpr int recv_bytes(int tn) { return tn == 64 ? 40960 : (tn <= 32 ? 32768 : 0); }

template <int FMT, int CG, int TN>
struct Cfg {
  static constexpr bool MX = FMT == kG8MX;
  static constexpr int STEP = 16 * CG;
  static constexpr int XROWS = TN / CG;  // rows of x staged per CTA
  static constexpr int X_BYTES = XROWS * BK;
  static constexpr int EPI_WARPS = TN >= 128 ? 8 : 4;
  static constexpr int EPI_COLS = TN / (EPI_WARPS / 4);  // columns per epilogue warp
  static constexpr int SC_WARPS = MX ? 4 : 1;       // warps that prepare scales
  static constexpr int EPI_FIRST = MX ? 8 : 4;       // first epilogue warp
  // MXFP8 on pairs: two sets of scale warps, each every other stage (a stage's chain
  // of load, tensor-memory store and its completion is longer than its MMAs)
  static constexpr int SC_SETS = MX && CG == 2 ? 2 : 1;
  static constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS + (SC_SETS - 1) * SC_WARPS);
  static constexpr int SF_BYTES = MX ? kAtomBytes : 0;  // weight scales of a stage
  static constexpr int SLOTS = MX ? 0 : 8;              // fp8_128: blocks of K whose scales are staged
  static constexpr int RECV_BYTES = CG == 1 ? recv_bytes(TN) : 0;
  static constexpr int FIXED = SLOTS * TN * 4 + RECV_BYTES + EPI_WARPS * 1024 + (3 * kMaxGroups + 1) * 4 + 512;
  static constexpr int FIT = (232448 - 1024 - FIXED) / (W_BYTES + X_BYTES + SF_BYTES);
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int OFF_W = 0;
  static constexpr int OFF_X = OFF_W + STAGES * W_BYTES;
  static constexpr int OFF_SFW = OFF_X + STAGES * X_BYTES;
  static constexpr int OFF_RECV = OFF_SFW + STAGES * SF_BYTES;
  static constexpr int OFF_SC = OFF_RECV + RECV_BYTES;
  static constexpr int OFF_OUT = OFF_SC + SLOTS * TN * 4;
  static constexpr int OFF_TABLE = OFF_OUT + EPI_WARPS * 1024;
  static constexpr int OFF_BAR = (OFF_TABLE + (3 * kMaxGroups + 1) * 4 + 7) / 8 * 8;
  // tensor memory: MXFP8 two accumulators (on pairs overlapping from column 128
  // on) and a slot of scales a stage; fp8_128 a ring of sums of one block of K
  static constexpr int ACOLS = TN < 32 ? 32 : TN;
  static constexpr bool OVERLAP = MX && CG == 2;
  static constexpr int BUFS = MX ? 2 : 4;
  static constexpr int ACC_STEP = OVERLAP ? 128 : ACOLS;
  static constexpr int T_SF = OVERLAP ? 384 : 2 * ACOLS;
  static constexpr int SFX_COLS = TN > 128 ? 8 : 4;
  static constexpr int SLOT_COLS = 4 + SFX_COLS;
  static constexpr int T_END = MX ? T_SF + STAGES * SLOT_COLS : BUFS * ACOLS;
  static constexpr int TMEM_COLS = T_END <= 128 ? 128 : (T_END <= 256 ? 256 : 512);
  static_assert(T_END <= 512 && (MX || CG == 1), "tensor memory");
  // barriers: full, empty; MXFP8 sf_full, sf_ready a stage; buf_full (MXFP8), buf_free a
  // buffer; sc_full, sc_free a slot; received.  fp8_128: the commit that frees a stage
  // also says that the block's sums are there (one commit a block less: M = 1, N = 2048,
  // K = 4096 5.7 -> 5.5 us); a stage's next phase is further off than the buffers reach.
  static constexpr int NBARS = (MX ? 4 : 2) * STAGES + 2 * BUFS + 2 * SLOTS + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 232448 && STAGES >= (MX ? 4 : BUFS + 1), "shared memory");
};

// ---------------------------------------------------------------- fragments
// 16 lanes x 8 NG columns: thread t receives, of group g of 8 columns, r[4g],
// r[4g+1] = lane t/4, columns 2 (t%4) and the next; r[4g+2], r[4g+3] = lane t/4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Four 8 x 8 tiles of 16-bit values, transposed on the way to shared memory: lane
// i gives the address of row i % 8 of tile i / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t m0, uint32_t m1, uint32_t m2, uint32_t m3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(m0), "r"(m1),
               "r"(m2), "r"(m3)
               : "memory");
}

// a += p * s; volatile, so that it stays behind the wait for p's load
__device__ __forceinline__ void add_scaled(float& a, uint32_t p, float s) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(a) : "f"(__uint_as_float(p)), "f"(s));
}

__device__ __forceinline__ void st_async_v4(uint32_t addr, float a, float b, float c, float d, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(__float_as_uint(d)), "r"(bar)
               : "memory");
}

// kQuant: few rows of bf16 x of one group, quantised here (fp8_128): four more warps
// load each stage's rows and write the codes where TMA would have put them and the
// scales where warp 3 would, the bytes of the quantise kernel.  That saves a launch, a
// workspace and the way through memory.
constexpr int QUANT_WARPS = 4;
constexpr int QUANT_ROWS = 8;

template <int FMT, int CG, int TN, bool kQuant>
constexpr int threads_of() {
  return Cfg<FMT, CG, TN>::THREADS + (kQuant ? 32 * QUANT_WARPS : 0);
}

template <int FMT, int CG, int TN, bool kQuant>
__global__ void __launch_bounds__(threads_of<FMT, CG, TN, kQuant>(), 1)
    gemm_grouped_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmXbox, const Args a) {
  using C = Cfg<FMT, CG, TN>;
  constexpr bool MX = C::MX;
  constexpr int STAGES = C::STAGES, BUFS = C::BUFS, SLOTS = C::SLOTS, STEP = C::STEP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* sf_full = empty + STAGES;                       // MXFP8
  uint64_t* sf_ready = sf_full + (MX ? STAGES : 0);         // MXFP8
  uint64_t* buf_full = sf_ready + (MX ? STAGES : 0);
  uint64_t* buf_free = buf_full + BUFS;
  uint64_t* sc_full = buf_free + BUFS;                      // fp8_128
  uint64_t* sc_free = sc_full + SLOTS;
  uint64_t* received = sc_free + SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  GroupTable table;
  table.start = reinterpret_cast<int*>(smem + C::OFF_TABLE);
  table.count = table.start + kMaxGroups;
  table.before = table.count + kMaxGroups;

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_ctarank());
  const int csize = CG == 2 ? 2 : a.splits;
  const int rank = CG == 2 ? cta & 1 : 0;  // in the pair
  const bool leader = rank == 0;
  const int worker = static_cast<int>(blockIdx.x) / csize, nworkers = static_cast<int>(gridDim.x) / csize;
  const int kt0 = CG == 2 ? 0 : cta * a.KT / a.splits;
  const int kt1 = CG == 2 ? a.KT : (cta + 1) * a.KT / a.splits;

  if (warp == 0) {
    for (int i = lane; i < C::NBARS; i += 32) {
      uint32_t n = 1;
      uint64_t* b = &full[i];
      if (kQuant && b < empty) n = 1 + a.R;  // the copies, and each row's codes
      if (MX && b >= sf_ready && b < buf_full) n = CG * C::SC_WARPS;
      if (b >= buf_free && b < sc_full) n = CG * C::EPI_WARPS;
      if (!MX && b >= sc_full && b < sc_free) n = kQuant ? a.R : C::SC_WARPS;
      if (!MX && b >= sc_free && b < received) n = C::EPI_WARPS;
      mbar_init(b, n);
    }
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
    __syncwarp();
  }
  // The weights of stage s at K tile kt of tile t, and what the stage waits for.  Both
  // CTAs' operands complete on the even CTA's `full`, whose bytes the even CTA alone
  // posts.  (They may land before the post, not a phase early: the stage was freed by
  // a commit behind the MMA that waited for the last phase.)
  const uint32_t base = smem_u32(smem);
  const uint32_t elected = elect_one();
  auto load_weights = [&](int s, int kt, const Tile& t) {
    const int rt = t.wt * CG + rank;
    const uint32_t bar = (CG == 2 ? map_shared_rank(smem_u32(full), 0) : smem_u32(full)) + s * 8;
    expect_tx(leader ? elected : 0u, &full[s], CG * W_BYTES + (kQuant ? 0 : t.width * BK));
    tma_load<CG>(elected, base + C::OFF_W + s * W_BYTES, &tmW, bar, kt * BK, rt * ROWS, t.e);
    if (MX && elected) {
      mbar_arrive_expect_tx(&sf_full[s], kAtomBytes);
      bulk_load(smem + C::OFF_SFW + s * C::SF_BYTES,
                static_cast<const uint8_t*>(a.ws) +
                    ((static_cast<int64_t>(t.e) * a.KT + kt) * a.RTW + min(rt, a.RTW - 1)) * kAtomBytes,
                kAtomBytes, &sf_full[s]);
    }
    __syncwarp();
  };
  // Without offsets (fp8_128 alone) the first round of weights needs nothing but this
  // warp's barriers (one CTA a tile; on a pair, the other CTA's too).
  int early = 0;
  if (!MX && CG == 1 && warp == 0 && a.offsets == nullptr && worker < unit_count<TN>(a, table)) {
    const Tile t = tile_of<STEP, TN>(worker, a, table);
    early = min(STAGES, kt1 - kt0);
    for (int s = 0; s < early; ++s) load_weights(s, kt0 + s, t);
  }
  if (threadIdx.x == 96) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmXbox);
  }
  if (warp == 1) {
    if (CG == 2) {
      tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  if (a.offsets != nullptr) {
    if (!a.offsets_ready) grid_dependency_wait();
    load_offsets(a, table, threads_of<FMT, CG, TN, kQuant>());
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (a.offsets != nullptr) {
    if (warp == 3) fill_table<TN>(a, table, lane);
    __syncthreads();
  }
  if (csize > 1) {
    cluster_arrive_relaxed();
    cluster_wait();  // every CTA's barriers exist before anyone signals them
  }
  if (CG == 1) launch_dependents();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const int units = unit_count<TN>(a, table);

  if (warp < 4) {
    if (warp == 0 || (warp == 2 && !kQuant)) {
      // ------------------------------------------------------------ producers
      const uint32_t full_bar = CG == 2 ? map_shared_rank(smem_u32(full), 0) : smem_u32(full);
      if (warp == 2) grid_dependency_wait();
      // Behind the weights that are on their way since the start.  (Their stages are not
      // waited for: the MMAs of one may be over before this warp comes by, and its next
      // phase waits for this warp.)
      int stage = early % STAGES, kt = kt0 + early;
      uint32_t phase = early < STAGES ? 1 : 0;  // the first round's stages are free
      int64_t issued = early;
      bool ok = true;
      for (int u = worker; ok && u < units; u += nworkers, kt = kt0) {
        const Tile t = tile_of<STEP, TN>(u, a, table);
        const int mine = t.width / CG;  // rows of x this CTA stages
        const int x0 = t.row0 + rank * mine;
        for (; kt < kt1; ++kt, ++issued) {
          if (!mbar_wait_warp(&empty[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t bar = full_bar + stage * 8;
          if (warp == 0) {
            load_weights(stage, kt, t);
          } else if (mine == C::XROWS) {
            tma_load<CG>(elected, base + C::OFF_X + stage * C::X_BYTES, &tmX, bar, kt * BK, x0, 0);
          } else {
            for (int i = 0; i < mine; i += BOX)
              tma_load<CG>(elected, base + C::OFF_X + stage * C::X_BYTES + i * BK, &tmXbox, bar, kt * BK, x0 + i, 0);
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Before exit: every commit to this CTA's empty barriers has arrived, and with
      // it the copies that the MMAs before it waited for.
      if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
          if (issued <= s) continue;
          const int64_t last = (issued - 1 - s) / STAGES;
          mbar_wait(&empty[s], static_cast<uint32_t>(last & 1), nullptr);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer (even CTA)
      if (leader) {
        const uint64_t wd0 = sdesc_kmajor_sw128(base + C::OFF_W), xd0 = sdesc_kmajor_sw128(base + C::OFF_X);
        int stage = 0, n = 0;  // n: accumulators begun (MXFP8), blocks of K (fp8_128)
        uint32_t phase = 0;
        bool ok = true;
        for (int u = worker; ok && u < units; u += nworkers) {
          const Tile t = tile_of<STEP, TN>(u, a, table);
          // fp32 accumulation (MXFP8: UE8M0 scales), E4M3 operands, N >> 3 at bit 17, M >> 4 at bit 24
          const uint32_t idesc =
              MX ? idesc_mxf8(CG * ROWS, t.width)
                 : (1u << 4) | (static_cast<uint32_t>(t.width >> 3) << 17) | (static_cast<uint32_t>(CG * ROWS >> 4) << 24);
          uint32_t acc = 0;
          if (MX) {
            const int b = n & 1;
            acc = tmem + b * C::ACC_STEP;
            // overlapping accumulators: the last tile's shared columns are drained;
            // else the tile before that
            const bool wait = C::OVERLAP ? n > 0 : n > 1;
            if (wait && !mbar_wait_warp(&buf_free[C::OVERLAP ? b ^ 1 : b],
                                        static_cast<uint32_t>(((n - (C::OVERLAP ? 1 : 2)) >> 1) & 1), abort_flag)) {
              ok = false;
              break;
            }
          }
          for (int kt = kt0; kt < kt1; ++kt) {
            if ((MX && !mbar_wait_warp(&sf_ready[stage], phase, abort_flag)) ||
                !mbar_wait_warp(&full[stage], phase, abort_flag)) {
              ok = false;
              break;
            }
            if (!MX) {
              const int b = n % BUFS;
              acc = tmem + b * C::ACOLS;
              if (!mbar_wait_warp(&buf_free[b], static_cast<uint32_t>(((n / BUFS) & 1) ^ 1), abort_flag)) {
                ok = false;
                break;
              }
            }
            tc_fence_after();
            const uint64_t wd = wd0 + static_cast<uint32_t>(stage * (W_BYTES >> 4));
            const uint64_t xd = xd0 + static_cast<uint32_t>(stage * (C::X_BYTES >> 4));
            const uint32_t t_sfw = tmem + C::T_SF + stage * C::SLOT_COLS;
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk) {
              if (MX)
                mma_mxf8<CG>(elected, acc, wd + 2 * kk, xd + 2 * kk, idesc_with_sf_id(idesc, kk, kk), t_sfw, t_sfw + 4,
                             ((kt - kt0) | kk) != 0);
              else
                mma_f8<CG>(elected, acc, wd + 2 * kk, xd + 2 * kk, idesc, kk != 0);
            }
            commit<CG>(elected, &empty[stage]);
            if (!MX) ++n;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (MX) {
            commit<CG>(elected, &buf_full[n & 1]);
            ++n;
          }
        }
        if (!ok) __nanosleep(200000);  // let issued tensor-core work retire
      }
      __syncwarp();
    } else if (!MX && !kQuant && warp == 3) {
      // ---------------------------------------------------------- fp8_128: s_x s_w of a block of K and each row of x
      // Lane l prepares rows l, l + 32, ...  Column c = 16 J + 8 g + 2 q + b goes to
      // position 16 J + 4 q + 2 g + b: 16 bytes are what a thread of the epilogue
      // (q) needs for 16 columns.
      constexpr int NR = TN < 32 ? 1 : TN / 32;
      grid_dependency_wait();  // x's scales are the previous kernel's output
      const int pos = (lane & ~15) | ((lane & 6) << 1) | ((lane & 8) >> 2) | (lane & 1);
      float* slots = reinterpret_cast<float*>(smem + C::OFF_SC);
      int slot = 0;
      uint32_t phase = 1;
      bool ok = true;
      float x[NR] = {}, w = 0.f;  // of the block ahead
      int f_u = worker, f_kt = kt0, f_rows = 0;
      const float *f_x = nullptr, *f_w = nullptr;
      auto start = [&]() {
        if (f_u >= units) return;
        const Tile t = tile_of<STEP, TN>(f_u, a, table);
        f_rows = t.rows;
        f_x = reinterpret_cast<const float*>(a.xs) + static_cast<int64_t>(t.row0 + lane) * a.xs_row + kt0 * a.xs_kt;
        const int rt = min(t.wt * CG + rank, a.RTW - 1);
        f_w = static_cast<const float*>(a.ws) + (static_cast<int64_t>(t.e) * a.RTW + rt) * a.KT + kt0;
      };
      auto fetch = [&]() {
        if (f_u >= units) return;
        w = __ldg(f_w++);
#pragma unroll
        for (int i = 0; i < NR; ++i) x[i] = lane + 32 * i < f_rows ? __ldg(f_x + 32 * i * a.xs_row) : 0.f;
        f_x += a.xs_kt;
        if (++f_kt == kt1) {
          f_kt = kt0;
          f_u += nworkers;
          start();
        }
      };
      start();
      fetch();
      for (int u = worker; ok && u < units; u += nworkers) {
        for (int kt = kt0; kt < kt1; ++kt) {
          if (!mbar_wait_warp(&sc_free[slot], phase, abort_flag)) {
            ok = false;
            break;
          }
          if (TN >= 32 || lane < TN) {
#pragma unroll
            for (int i = 0; i < NR; ++i) slots[slot * TN + pos + 32 * i] = x[i] * w;
          }
          fetch();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[slot]);
          if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (MX && (warp < 8 || warp >= C::EPI_FIRST + C::EPI_WARPS)) {
    grid_dependency_wait();  // x's scales are the previous kernel's output
    // ---------------------------------------------------------- MXFP8 scales into tensor memory
    // Line l of an atom (rows l, l + 32, l + 64, l + 96) goes to lane l of each
    // quarter, one quarter a warp.  The words of x's rows are loaded AHEAD stages early.
    constexpr int NW = TN < 32 ? 1 : TN / 32, AHEAD = 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::T_SF;
    const uint32_t ready = CG == 2 ? map_shared_rank(smem_u32(sf_ready), 0) : smem_u32(sf_ready);
    constexpr int SETS = C::SC_SETS;
    const int set = warp < 8 ? 0 : 1, nk = kt1 - kt0;
    int f_u = worker, f_kt = kt0 + set, f_rows = 0;
    const uint32_t* f_p = a.xs;
    auto start = [&]() {  // the tile that stage f_kt counted from f_u's first falls into
      while (f_kt >= kt1 && f_u < units) {
        f_kt -= nk;
        f_u += nworkers;
      }
      if (f_u >= units) return;
      const Tile t = tile_of<STEP, TN>(f_u, a, table);
      f_rows = t.rows - lane;
      f_p = a.xs + static_cast<int64_t>(t.row0 + lane) * a.xs_row + f_kt * a.xs_kt;
    };
    start();
    auto fetch = [&](uint32_t (&w)[NW]) {
      if (f_u >= units) return;
#pragma unroll
      for (int i = 0; i < NW; ++i) w[i] = 32 * i < f_rows ? __ldg(f_p + 32 * i * a.xs_row) : 0u;
      f_p += SETS * a.xs_kt;
      f_kt += SETS;
      if (f_kt >= kt1) start();
    };
    uint32_t w[AHEAD][NW] = {};
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) fetch(w[d]);
    int stage = set;
    uint32_t phase = 0;
    bool ok = true;
    int64_t left = -set;  // stages of this set
    for (int u = worker; u < units; u += nworkers) left += nk;
    left = (left + SETS - 1) / SETS;
    while (ok && left > 0) {
#pragma unroll
      for (int d = 0; d < AHEAD; ++d, --left) {
        if (!ok || left <= 0) break;
        // the stage's slot is free: its refill has waited for the MMAs that read it
        if (!mbar_wait_warp(&sf_full[stage], phase, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint4 v = reinterpret_cast<const uint4*>(smem + C::OFF_SFW + stage * C::SF_BYTES)[lane];
        const uint32_t ts = lane_base + stage * C::SLOT_COLS;
        tmem_st_32x32b_x4(ts, v.x, v.y, v.z, v.w);
#pragma unroll
        for (int i = 0; i < NW; i += 4)
          tmem_st_32x32b_x4(ts + 4 + i, w[d][i], i + 1 < NW ? w[d][i + 1 < NW ? i + 1 : 0] : 0u,
                            i + 2 < NW ? w[d][i + 2 < NW ? i + 2 : 0] : 0u,
                            i + 3 < NW ? w[d][i + 3 < NW ? i + 3 : 0] : 0u);
        fetch(w[d]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!leader)
            mbar_arrive_remote(ready + static_cast<uint32_t>(stage * 8));
          else
            mbar_arrive(&sf_ready[stage]);
        }
        stage += SETS;
        if (stage >= STAGES) {
          stage -= STAGES;
          phase ^= 1u;
        }
      }
    }
  } else if (kQuant && warp >= C::EPI_FIRST + C::EPI_WARPS) {
    if constexpr (kQuant) {
      // ---------------------------------------------------------- quantisers
      // Eight lanes a task, a row of a stage: task i is row i % R of stage i / R,
      // counted on over this worker's units (one group of rows, so unit u is weight
      // tile u), and group g of up to 16 takes every groups-th.  From one task of a
      // group to its next are eight stages at the most, no more than there are stages
      // and slots: the place the next waits for has been freed up to the fill before
      // last, so that the wait's parity is right; and none waits for what a later task
      // of its warp would free.  A first round without effect, before x may be read,
      // brings the code into the instruction cache.
      static_assert(!MX && CG == 1 && TN == 16 && STAGES >= 8 && SLOTS >= 8, "few rows, fp8_128");
      const int group = (warp - C::EPI_FIRST - C::EPI_WARPS) * 4 + (lane >> 3);
      const int groups = min(4 * QUANT_WARPS, 8 * a.R), c = lane & 7;
      float* slots = reinterpret_cast<float*>(smem + C::OFF_SC);
      const int nk = kt1 - kt0;
      const int stages = units > worker ? ((units - 1 - worker) / nworkers + 1) * nk : 0;
      uint32_t v[8] = {};
      float w = 0.f;
      auto fetch = [&](int i) {
        const int at = i / a.R, r = i - at * a.R;
        const int nth = at / nk, st = kt0 + at - nth * nk, k = st * BK + 16 * c;
        const bool in = group < groups && at < stages;
        if (in) w = __ldg(static_cast<const float*>(a.ws) + static_cast<int64_t>(worker + nth * nworkers) * a.KT + st);
        if (in && k < a.K) {
          load16(a.x + static_cast<int64_t>(r) * a.K + k, false, v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = 0;
        }
      };
      // the warp's groups go round together; one without a task is idle
      const int last = (stages * a.R + groups - 1) / groups * groups;
      for (int i = group - groups; i < last; i += groups) {
        float scale;
        const Codes codes = quantize16_b128(v, &scale);
        const float sw = w;
        if (i < group) grid_dependency_wait();
        fetch(i + groups);
        const int at = i / a.R, r = i - at * a.R;
        const bool task = i >= 0 && group < groups && at < stages;
        const int stage = at % STAGES, slot = at % SLOTS;
        bool free = true;
        if (task)
          free = mbar_wait(&empty[stage], static_cast<uint32_t>((at / STAGES) & 1) ^ 1u, abort_flag) &&
                 mbar_wait(&sc_free[slot], static_cast<uint32_t>((at / SLOTS) & 1) ^ 1u, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, free)) break;
        if (task) {
          // 128-byte rows, 16-byte pieces swizzled as TMA does
          *reinterpret_cast<uint4*>(smem + C::OFF_X + stage * C::X_BYTES + r * BK + ((c ^ r) << 4)) =
              make_uint4(codes.w[0], codes.w[1], codes.w[2], codes.w[3]);
          if (c == 0) slots[slot * TN + (((r & 6) << 1) | (r & 1))] = scale * sw;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (task && c == 0) {
          mbar_arrive(&full[stage]);
          mbar_arrive(&sc_full[slot]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int COLS = C::EPI_COLS;
    constexpr int CH = COLS < 32 ? COLS : 32;  // columns per load
    constexpr int NCH = COLS / CH, NG = CH / 8;
    const int quad = warp & 3;
    const int ew = warp - C::EPI_FIRST;
    const int col_base = ew / 4 * COLS;
    uint8_t* box = smem + C::OFF_OUT + ew * 1024;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col_base;
    const uint32_t free_bar = CG == 2 ? map_shared_rank(smem_u32(buf_free), 0) : smem_u32(buf_free);
    auto release = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_remote(free_bar + static_cast<uint32_t>(b * 8));
        else
          mbar_arrive(&buf_free[b]);
      }
    };
    const uint32_t st_addr =
        smem_u32(box) + (lane & 7) * 64 + ((((lane >> 3) ^ (lane >> 1)) & 3) << 4);
    const uint8_t* ld_addr = box + (lane >> 2) * 64 + ((((lane & 3) ^ (lane >> 3)) & 3) << 4);
    int flip = 0;
    grid_dependency_wait();  // the bias may be the previous kernel's output
    // Eight columns (rows of x) of this warp's 32 weight rows, v[4 h ..] the fragment
    // of lanes 16 h ..: rounded, transposed, stored.
    Tile t;
    float bias[4];
    int n_lane = 0;
    auto start_tile = [&](int u) {
      t = tile_of<STEP, TN>(u, a, table);
      const int n0 = (t.wt * CG + rank) * ROWS + quad * 32;
      n_lane = n0 + (lane & 3) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 8 * i + (lane >> 2);
        bias[i] = a.bias != nullptr && n < a.N ? __bfloat162float(a.bias[t.e * a.bias_stride + n]) : 0.f;
      }
    };
    auto emit = [&](int col, const float (&v)[8]) {
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = pack_bf16x2(v[2 * i] + bias[i], v[2 * i + 1] + bias[i]);
      stmatrix_x4_trans(st_addr + flip, m[0], m[1], m[2], m[3]);
      __syncwarp();
      const uint4 o = *reinterpret_cast<const uint4*>(ld_addr + flip);
      const int r = col + (lane >> 2);
      if (r < t.rows && n_lane < a.N)
        *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(t.row0 + r) * a.N + n_lane) = o;
      flip ^= 512;  // the other half: this one is read before the next __syncwarp but one
    };
    // K splits: group j of 8 columns is finished by CTA j % S of the cluster; the
    // partial sums of all S go to its slot j / S, and are added in the order of K.
    float* recv = reinterpret_cast<float*>(smem + C::OFF_RECV);
    auto send = [&](int col, const float (&v)[8]) {
      const int j = col >> 3, S = a.splits;
      const int owner = j % S;
      float* at = recv + ((j / S * S + cta) * 4 + quad) * 256 + lane * 8;
      const uint32_t dst = map_shared_rank(smem_u32(at), owner);
      const uint32_t bar = map_shared_rank(smem_u32(received), owner);
      st_async_v4(dst, v[0], v[1], v[2], v[3], bar);
      st_async_v4(dst + 16, v[4], v[5], v[6], v[7], bar);
    };
    auto finish_split = [&]() {
      const int S = a.splits, groups = (t.rows + 7) >> 3;
      const int owned = groups > cta ? (groups - cta + S - 1) / S : 0;
      if (owned == 0) return;
      if (ew == 0 && lane == 0) mbar_arrive_expect_tx(received, static_cast<uint32_t>(owned * S * 4096));
      // waited for in any case: no store may land after this CTA has left
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(received, 0, nullptr))) return;
      for (int i = 0; i < owned; ++i) {
        float v[8] = {};
        for (int s = 0; s < S; ++s) {
          const float4* p = reinterpret_cast<const float4*>(recv + ((i * S + s) * 4 + quad) * 256 + lane * 8);
          const float4 p0 = p[0], p1 = p[1];
          v[0] += p0.x, v[1] += p0.y, v[2] += p0.z, v[3] += p0.w;
          v[4] += p1.x, v[5] += p1.y, v[6] += p1.z, v[7] += p1.w;
        }
        emit((i * S + cta) * 8, v);
      }
    };
    const bool split = CG == 1 && TN <= 64 && a.splits > 1;

    int n = 0;  // accumulators (MXFP8) or blocks of K (fp8_128) so far
    if constexpr (MX) {
      for (int u = worker; u < units; u += nworkers, ++n) {
        start_tile(u);
        const int b = n & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&buf_full[b], static_cast<uint32_t>((n >> 1) & 1), abort_flag))) {
          // without a sum of its own a CTA still waits for those of its cluster's others
          if (split) finish_split();
          break;
        }
        tc_fence_after();
        const uint32_t acc = lanes + b * C::ACC_STEP;
        // Pairs: the columns shared with the next tile's accumulator first (the
        // upper 128 of an even tile, the lower of an odd one); all eight warps
        // take 64 of those, then 64 of the others.
#pragma unroll 1
        for (int i = 0; i < NCH; ++i) {
          int at = i * CH;  // from col_base
          if (C::OVERLAP) {
            const int first = b ? 0 : 128;
            at = (i < NCH / 2 ? first : 128 - first) + col_base / 2 + (i & (NCH / 2 - 1)) * CH - col_base;
          }
          uint32_t r[2][4 * NG];
          if (at + col_base < t.width) {
            tmem_ld_frag(acc + at, r[0]);
            tmem_ld_frag(acc + at + (16u << 16), r[1]);
            tmem_ld_wait();
          }
          if (i == (C::OVERLAP ? NCH / 2 : NCH) - 1) release(b);
          if (at + col_base < t.width) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r[k >> 2][4 * g + (k & 3)]);
              const int col = col_base + at + 8 * g;
              if (col < t.rows) {
                if (split)
                  send(col, v);
                else
                  emit(col, v);
              }
            }
          }
        }
        if (split) finish_split();
      }
    } else {
      int slot = 0;
      uint32_t sphase = 0;
      for (int u = worker; u < units; u += nworkers) {
        float acc[NCH][2][4 * NG];  // as the fragments
#pragma unroll
        for (int i = 0; i < NCH * 8 * NG; ++i) (&acc[0][0][0])[i] = 0.f;
        // CH columns of all 32 lanes at a time (those that are not the tile's are added
        // like the others and not stored): the next ones are on their way while one lot
        // is added.
        constexpr int RB = NCH > 1 ? 2 : 1;
        uint32_t r[RB][2][4 * NG];
        float4 f[RB][CH / 16];
        auto load = [&](int i) {
          const uint32_t src = lanes + (n % BUFS) * C::ACOLS + i * CH;
          tmem_ld_frag(src, r[i % RB][0]);
          tmem_ld_frag(src + (16u << 16), r[i % RB][1]);
          const float4* sc =
              reinterpret_cast<const float4*>(smem + C::OFF_SC) + (slot * TN + col_base + i * CH) / 4 + (lane & 3);
#pragma unroll
          for (int k = 0; k < CH / 16; ++k) f[i % RB][k] = sc[4 * k];
        };
        for (int kt = kt0; kt < kt1; ++kt) {
          // the sums of block n (in buffer n % BUFS) and its scales; a wait that ran out
          // only makes the later ones return at once
          const uint32_t bp = static_cast<uint32_t>((n / STAGES) & 1);
          if (!mbar_try_wait(&sc_full[slot], sphase)) mbar_wait_inline(&sc_full[slot], sphase, abort_flag);
          if (!mbar_try_wait(&empty[n % STAGES], bp)) mbar_wait_inline(&empty[n % STAGES], bp, abort_flag);
          __syncwarp();
          tc_fence_after();
          load(0);
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            tmem_ld_wait();
            if (i + 1 < NCH) {
              load(i + 1);
            } else {
              release(n % BUFS);
              if (lane == 0) mbar_arrive(&sc_free[slot]);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              const float4 q = f[i % RB][g >> 1];
#pragma unroll
              for (int c = 0; c < 2; ++c) {  // the four sums of a column one after the other
                const float sc = g & 1 ? (c ? q.w : q.z) : (c ? q.y : q.x);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  add_scaled(acc[i][k >> 1][4 * g + 2 * (k & 1) + c], r[i % RB][k >> 1][4 * g + 2 * (k & 1) + c], sc);
              }
            }
          }
          ++n;
          if (++slot == SLOTS) {
            slot = 0;
            sphase ^= 1u;
          }
        }
        start_tile(u);
#pragma unroll
        for (int g = 0; g < COLS / 8; ++g) {
          const int col = col_base + 8 * g;
          if (col < t.rows) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = acc[g / NG][k >> 2][4 * (g % NG) + (k & 3)];
            if (split)
              send(col, v);
            else
              emit(col, v);
          }
        }
        if (split) finish_split();
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // No CTA of the cluster leaves while another may still signal it.  Pairs: the odd CTA's
  // last arrivals on buf_free are waited for by nobody, so this barrier has to order them.
  // K splits: all that is sent is waited for above.
  if (CG == 2) {
    cluster_sync();
  } else if (csize > 1) {
    cluster_arrive_relaxed();
    cluster_wait();
  }
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2)
      tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else
      tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int FMT, int CG, int TN, bool kQuant = false>
cudaError_t launch_t(const GroupedProblem& p, int splits, int sms, cudaStream_t stream, const char** msg) {
  using C = Cfg<FMT, CG, TN>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaError_t e =
        cudaFuncSetAttribute(gemm_grouped_kernel<FMT, CG, TN, kQuant>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) {
      *msg = "cudaFuncSetAttribute(max dynamic shared memory) failed";
      return e;
    }
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  CUtensorMap mw, mx, mbox;
  if (!grouped_maps(p, kQuant ? 0 : C::XROWS, &mw, &mx, &mbox)) {
    *msg = "cuTensorMapEncodeTiled rejected an operand of the grouped product";
    return cudaErrorInvalidValue;
  }
  const Args a = grouped_args(p, CG, splits);
  const int64_t units = grouped_max_tiles(p.E, p.R, p.offsets != nullptr, TN) * a.WT;
  const int csize = CG == 2 ? 2 : splits;
  int64_t workers = splits > 1 ? units : (units < sms / CG ? units : sms / CG);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(workers * csize), 1, 1);
  cfg.blockDim = dim3(threads_of<FMT, CG, TN, kQuant>(), 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(csize);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_grouped_kernel<FMT, CG, TN, kQuant>, mw, mx, mbox, a);
  if (e != cudaSuccess) *msg = "grouped product launch failed";
  return e;
}

template <int FMT>
cudaError_t launch_fmt(const GroupedProblem& p, const GroupedPlan& plan, int sms, cudaStream_t stream,
                       const char** msg) {
  if (plan.cg == 2) {
    if constexpr (FMT == kG8MX)
      return launch_t<FMT, 2, 256>(p, 1, sms, stream, msg);
    else
      return launch_gemm_b128_pair(p, sms, stream, msg);
  }
  if constexpr (FMT == kG8B128) {
    if (p.x_bf16 != nullptr) return launch_t<FMT, 1, 16, true>(p, plan.splits, sms, stream, msg);
  }
  if (plan.tn == 16) return launch_t<FMT, 1, 16>(p, plan.splits, sms, stream, msg);
  if (plan.tn == 32) return launch_t<FMT, 1, 32>(p, plan.splits, sms, stream, msg);
  if (plan.tn == 64) return launch_t<FMT, 1, 64>(p, plan.splits, sms, stream, msg);
  return launch_t<FMT, 1, 128>(p, 1, sms, stream, msg);
}

}  // namespace

// Tensor maps of the weights, and of x in boxes of box_rows and of kGBox rows.
bool grouped_maps(const GroupedProblem& p, int box_rows, CUtensorMap* mw, CUtensorMap* mx, CUtensorMap* mbox) {
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const auto l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if (!encode_map3(mw, u8, p.w, p.K, p.N, p.E, p.K, p.N * p.K, kGBK, kGW_Rows, sw, l2)) return false;
  if (box_rows == 0) {  // x is not copied
    *mx = *mbox = *mw;
    return true;
  }
  return encode_map3(mbox, u8, p.x, p.K, p.R, 1, p.K, p.R * p.K, kGBK, kGBox, sw, l2) &&
         (box_rows == kGBox ? (*mx = *mbox, true)
                            : encode_map3(mx, u8, p.x, p.K, p.R, 1, p.K, p.R * p.K, kGBK, box_rows, sw, l2));
}

GroupedArgs grouped_args(const GroupedProblem& p, int cg, int splits) {
  GroupedArgs a;
  a.offsets = p.offsets;
  a.groups = static_cast<int>(p.E);
  a.M = p.offsets != nullptr ? 0 : static_cast<int>(p.R / p.E);
  a.R = static_cast<int>(p.R);
  a.N = static_cast<int>(p.N);
  a.WT = static_cast<int>(ceil_div(p.N, cg * kGW_Rows));
  a.KT = static_cast<int>(ceil_div(p.K, kGBK));
  a.splits = splits;
  a.offsets_ready = p.offsets_ready;
  a.w_fast = p.R / p.E >= p.N ? 1 : 0;
  a.xs = static_cast<const uint32_t*>(p.xs);
  a.xs_row = p.xs_row;
  a.xs_kt = p.xs_kt;
  a.ws = p.ws;
  a.RTW = static_cast<int>(ceil_div(p.N, kGW_Rows));
  a.bias = static_cast<const __nv_bfloat16*>(p.bias);
  a.bias_stride = p.bias_stride;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.x = static_cast<const __nv_bfloat16*>(p.x_bf16);
  a.K = static_cast<int>(p.K);
  return a;
}

int64_t grouped_max_tiles(int64_t E, int64_t R, bool ragged, int tn) {
  if (!ragged) return E * ceil_div(R / E, tn);
  return (E < R ? E : R) + R / tn;
}

namespace {

// The counts below are GB300's: 152 SMs, 76 pairs, the clusters that fit at once.  With
// others the choice is slower, never wrong: no kernel needs its CTAs to run together
// but for the clusters.
// Estimated time of a shape on one CTA a tile with up to tn rows of x and K split s
// ways, or on pairs (tn = 256), in 0.01 us.  Measured (us, fp8_128, weights from HBM;
// the quantise kernel and the launches, 6 to 8, included): a stage of K takes 0.24 to
// 0.26 with up to 64 rows, 0.36 with 128 and on pairs; N = K = 4096, M = 1, one to
// eight splits 13.7 / 11.0 / 10.9 / 21.6 (two waves of clusters); M = 200, 64 rows a
// tile 17.6, 128 20.5, pairs 23.0; M = 512 25.9 / 20.2 / 20.3; N = 14336, K = 4096,
// M = 48 18.6 / 18.7 / 22.0, M = 256 34.6 / 31.1 / 22.1; N = 1000, K = 4096, M = 333,
// 64 rows and two splits 15.1, one 16.2, 128 rows 20.1, pairs 22.3.  A split costs the
// exchange, more of it in larger clusters, and once two calls in a row do not fit the
// SMs together their overlap; pairs start 2 us later.  Over 1500 shapes, 1 to 24576
// rows, the choice took 2.0 % more time on average than the best that was tried (5 % of
// them 10 to 36 %, most of those with few of the experts at work).
int64_t plan_cost(int64_t groups, int64_t rows, int64_t N, int64_t K, int tn, int splits) {
  const int64_t stages = ceil_div(K, kGBK);
  const int64_t workers = tn == 256 ? 76 : 152;
  const int64_t tiles = groups * ceil_div(rows, tn) * ceil_div(N, tn == 256 ? 256 : 128) * splits;
  const int64_t stage = tn == 256 ? 40 : (tn == 128 ? 36 : (tn == 64 ? 26 : 24));
  const int64_t tile = stage * ceil_div(stages, splits) + (splits > 1 ? 150 + 20 * splits + tn + (tiles > 76 ? 60 : 0) : (tn == 256 ? 130 : 150));
  const int64_t bytes = groups * N * K / 65000;  // the weights at 6.5 TB/s
  const int64_t t = ceil_div(tiles, workers) * tile + (tn == 256 ? 200 : 0);
  return t > bytes ? t : bytes + tn;  // bound by the weights: the narrowest
}

}  // namespace

bool b128_quantizes_inside(bool ragged, int64_t E, int64_t R) { return !ragged && E == 1 && R <= QUANT_ROWS; }

// With offsets the host knows the rows a group has only on average, and groups
// without rows only where there are fewer rows than groups: it counts on twice as many,
// because a tile that is too wide costs less than a second one (108 experts, 55 of them
// with the 1416 rows, 1216 x 1744, fp8_128, 64 rows a tile 27.5 us, 16, enough for the
// average, 37.0).
GroupedPlan grouped_plan(int fmt, int64_t E, int64_t R, int64_t N, int64_t K, bool ragged) {
  const int64_t groups = E < R ? E : (R > 0 ? R : 1), mean = ceil_div(R, groups), rows = ragged && mean > 1 ? 2 * mean : mean;
  const bool few = fmt == kG8B128 && b128_quantizes_inside(ragged, E, R);
  GroupedPlan best = {2, 256, 1};
  int64_t least = few ? INT64_MAX : plan_cost(groups, rows, N, K, 256, 1);
  for (int tn = few ? 16 : 128; tn >= 16; tn >>= 1) {
    // at most eight tiles of x a group, unless all tiles run at once: each reads the
    // weights again, from L2
    const int64_t tiles = ceil_div(rows, tn);
    if (tiles > 8 && groups * tiles * ceil_div(N, kGW_Rows) > 152) break;
    for (int s = 1; s <= 8; ++s) {
      // split, a cluster does one tile: all of them, however the rows fall, at once.
      // kClusterSMs: one cluster less than the occupancy calculator has room for (M = 64, N
      // = 2048, K = 16384, 128 CTAs in clusters of 8 20.0 us, of 4 13.0, of 5 12.4; M = 1,
      // N = 2048, K = 4096 clusters of 8 10.4, of 4 5.6; M = 16, N = K = 5120 clusters of
      // 2 8.3, of 3 7.6).  Of 7 there are no more than of 8.
      constexpr int kClusterSMs[9] = {0, 152, 152, 135, 140, 135, 132, 0, 112};
      if (s > 1 && (received_bytes(tn, s) > recv_bytes(tn) || ceil_div(K, kGBK) < 2 * s ||
                    grouped_max_tiles(E, R, ragged, tn) * ceil_div(N, kGW_Rows) * s > kClusterSMs[s]))
        continue;
      const int64_t c = plan_cost(groups, rows, N, K, tn, s);
      if (c <= least) {
        least = c;
        best = {1, tn, s};
      }
    }
  }
  return best;
}

cudaError_t launch_gemm_grouped(const GroupedProblem& p, const GroupedPlan& plan, int sms, cudaStream_t stream,
                                const char** msg) {
  return p.fmt == kG8MX ? launch_fmt<kG8MX>(p, plan, sms, stream, msg) : launch_fmt<kG8B128>(p, plan, sms, stream, msg);
}

cudaError_t take_status_grouped(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
}

}  // namespace mx
