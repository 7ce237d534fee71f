// gemm_b128_pair.cu - the block-128 FP8 product on CTA pairs, for groups of more
// rows than the one-CTA kernel of gemm_grouped.cu is for:
//   out[r, n] = bf16( sum_j s_x[r, j] s_w[e, n / 128, j] sum_(k in block j) x w + bias )
// tcgen05.mma kind::f8f6f4 sums one block of 128 along K in tensor memory, and the
// epilogue warps add it to fp32 registers times its scale.
//
// Here the rows of x are the MMA's M side: a thread then holds one row, and its
// scale s_x s_w is one number for a whole block of K.  (With the weights on the M
// side, as for MXFP8, ragged rows leave no MMA column unused, but each
// multiply-add reads a sum, an addend and a scale of its own from the register
// file, which delivers two operands a cycle: 128 of them a warp, two warps a
// scheduler, take 412 cycles a block where a scale that stays takes 262, and the
// scales have to be read from shared memory by every warp.  M = 4096, N = 14336, K
// = 4096 took 271 us so.)
//
// Bound by the round of the two buffers: 512 cycles of MMAs, their commit, the load
// of a buffer into registers (its first half is added before the second has room)
// and the way back to the MMA warp, ~0.85 us for two blocks, a little over what the
// operands need from L2 (0.37 us a block) and the multiply-adds of two warps a
// scheduler (~320 cycles).  M = 4096, N = 14336, K = 4096 168 us, 2.9 PFLOP/s, tensor
// pipe 61 % busy (ncu), issue slots 57 %; 24576 rows on 61 of 64 experts of 4096 x
// 2048 229 us: 16 blocks a tile, and a tile's start and output cost 1.3 us more.
// Steps, the first of those shapes: rows of x in lanes 231 -> scales loaded by the
// thread that needs them 214 -> output through shared memory 210 -> no branch on the
// tile in the loop 179 -> the wait for the next block after the additions 172 -> 64
// columns at a time, the buffer given back before the last are added 166.  Not kept:
// the columns as two MMAs of 128 with a barrier each, so that the two warps of a
// scheduler come apart (273; what of it the narrower MMAs cost and what the second
// barrier was not told apart); test_wait spins (+0); the next tile's first scales
// before the output (+1 %); a group's last tile of up to 128 rows with the weights on
// the M side and its rows in as few columns as hold them (64 groups of 272 rows, N = K =
// 2048, 115 instead of 119 us, of 384 rows 143 instead of 120).
//
// A cluster of two CTAs computes 256 rows x 256 weight rows with cta_group::2: CTA r
// stages rows [128 r, +128) of both tiles and receives the sums of its rows of x.
// Where a group's last tile has at most 128 rows, the odd CTA loads one box of rows
// and adds nothing.  Warps: 0 weight TMA, 1 tensor-memory allocation and (even CTA) MMA
// issue, 2 TMA of x, 3 the group table, 4..11 epilogue (128 sums a thread, so the
// registers are split unevenly).  Every wait is bounded and the
// cluster barriers are reached on every path.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_grouped.cuh"
#include "mx_kernels.h"

namespace mx {

namespace {

constexpr int BM = 128;  // rows of x, and of the weights, per CTA
constexpr int BK = kGBK;
constexpr int TILE = 256;
constexpr int HALF_BYTES = BM * BK;
constexpr int STAGES = 6;
constexpr int BUFS = 2;   // tensor memory: sums of two blocks of K, 256 columns each
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int OFF_W = 0;
constexpr int OFF_X = OFF_W + STAGES * HALF_BYTES;
constexpr int OUT_BOX = 32 * 64;  // staging of an epilogue warp: 32 rows x 32 columns
constexpr int OFF_OUT = OFF_X + STAGES * HALF_BYTES;
constexpr int OFF_TABLE = OFF_OUT + EPI_WARPS * OUT_BOX;
constexpr int OFF_BAR = (OFF_TABLE + (3 * kMaxGroups + 1) * 4 + 7) / 8 * 8;
constexpr int NBARS = 2 * STAGES + 2 * BUFS;
constexpr int OFF_MISC = OFF_BAR + NBARS * 8;
constexpr int SMEM = OFF_MISC + 16 + 1024;
constexpr int TMEM_COLS = 512;
static_assert(SMEM <= 232448 && BUFS == 2, "shared memory; the epilogue flips between two buffers");

// a += p * s; volatile, so that it stays behind the wait for p's load
__device__ __forceinline__ void add_scaled(float& a, uint32_t p, float s) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(a) : "f"(__uint_as_float(p)), "f"(s));
}

__global__ void __launch_bounds__(THREADS, 1)
    gemm_b128_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmXbox, const GroupedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* buf_full = empty + STAGES;
  uint64_t* buf_free = buf_full + BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  GroupTable table;
  table.start = reinterpret_cast<int*>(smem + OFF_TABLE);
  table.count = table.start + kMaxGroups;
  table.before = table.count + kMaxGroups;

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank() & 1u);
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);

  if (warp == 0) {
    for (int i = lane; i < NBARS; i += 32) {
      mbar_init(&full[i], &full[i] >= buf_free ? 2 * EPI_WARPS : 1);
    }
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 96) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmXbox);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (a.offsets != nullptr) {
    if (!a.offsets_ready) grid_dependency_wait();
    load_offsets(a, table, THREADS);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (a.offsets != nullptr) {
    if (warp == 3) fill_table<TILE>(a, table, lane);
    __syncthreads();
  }
  cluster_arrive_relaxed();
  cluster_wait();  // both CTAs' barriers exist before anyone signals them
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const int units = unit_count<TILE>(a, table);
  const uint32_t base = smem_u32(smem);

  // 168 registers a thread at the launch: 40 + 2 * 232 = 3 * 168
  if (warp < 4) {
    set_registers_dec<40>();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- producers
      // Both CTAs' operands complete on the even CTA's `full`, whose bytes the even
      // CTA alone posts.  (They may land before the post, not a phase early: the
      // stage was freed by a commit behind the MMA that waited for the last phase.)
      const uint32_t elected = elect_one();
      const uint32_t poster = leader ? elected : 0u;
      const uint32_t full_bar = map_shared_rank(smem_u32(full), 0);
      if (warp == 2) grid_dependency_wait();
      int stage = 0;
      uint32_t phase = 1;  // the first round's stages are free
      int64_t issued = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += npairs) {
        const GroupTile t = tile_of<0, TILE>(u, a, table);
        // Rows of x that the CTAs stage, whole boxes; what a stage holds behind them
        // only goes into sums that are not stored.  At least one box each, even of
        // rows that are not the tile's: `full` has to depend on both CTAs' warp 2.
        // Left out of the round, it could fall behind by two phases of `empty`,
        // whose parity it would then misread, and wait for good.
        const int rows0 = (min(t.rows, BM) + kGBox - 1) / kGBox * kGBox;
        const int rows1 = (max(t.rows - BM, 1) + kGBox - 1) / kGBox * kGBox;
        const int mine = rank ? rows1 : rows0, x0 = t.row0 + rank * BM;
        const uint32_t bytes = static_cast<uint32_t>(2 * HALF_BYTES + (rows0 + rows1) * BK);
        for (int kt = 0; kt < a.KT; ++kt, ++issued) {
          if (!mbar_wait_warp(&empty[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t bar = full_bar + stage * 8;
          if (warp == 0) {
            expect_tx(poster, &full[stage], bytes);
            tma_load<2>(elected, base + OFF_W + stage * HALF_BYTES, &tmW, bar, kt * BK, t.wt * TILE + rank * BM, t.e);
          } else if (mine == BM) {
            tma_load<2>(elected, base + OFF_X + stage * HALF_BYTES, &tmX, bar, kt * BK, x0, 0);
          } else {
            for (int i = 0; i < mine; i += kGBox)
              tma_load<2>(elected, base + OFF_X + stage * HALF_BYTES + i * BK, &tmXbox, bar, kt * BK, x0 + i, 0);
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
          mbar_wait(&empty[s], static_cast<uint32_t>(((issued - 1 - s) / STAGES) & 1), nullptr);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer (even CTA)
      if (leader) {
        // E4M3 operands, fp32 sums, N >> 3 at bit 17, M >> 4 at bit 24
        constexpr uint32_t idesc = (1u << 4) | ((TILE >> 3) << 17) | ((TILE >> 4) << 24);
        const uint32_t elected = elect_one();
        const uint64_t wd0 = sdesc_kmajor_sw128(base + OFF_W), xd0 = sdesc_kmajor_sw128(base + OFF_X);
        int stage = 0, b = 0;
        uint32_t phase = 0, bphase = 1;
        bool ok = true;
        for (int u = pair; ok && u < units; u += npairs) {
          for (int kt = 0; kt < a.KT; ++kt) {
            if (!mbar_wait_warp(&full[stage], phase, abort_flag) || !mbar_wait_warp(&buf_free[b], bphase, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t wd = wd0 + static_cast<uint32_t>(stage * (HALF_BYTES >> 4));
            const uint64_t xd = xd0 + static_cast<uint32_t>(stage * (HALF_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              mma_f8<2>(elected, tmem + b * TILE, xd + 2 * kk, wd + 2 * kk, idesc, kk != 0);
            commit<2>(elected, &buf_full[b]);
            commit<2>(elected, &empty[stage]);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            if (++b == BUFS) {
              b = 0;
              bphase ^= 1u;
            }
          }
        }
        if (!ok) __nanosleep(200000);  // let issued tensor-core work retire
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Warp e: rows 32 (e % 4).. of the CTA, columns [128 (e / 4), +128): one block of
    // the weights.
    set_registers_inc<232>();
    const int ew = warp - 4, half = ew >> 2;
    const int my_row = (warp & 3) * 32 + lane;  // in the CTA
    const uint32_t src = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * 128;
    const uint32_t free_bar = map_shared_rank(smem_u32(buf_free), 0);
    grid_dependency_wait();  // x's scales and the bias may be the previous kernel's output
    int b = 0;
    uint32_t bphase = 0;
    // The loop below runs at the pace of its instructions: two warps a scheduler, 128
    // multiply-adds a block and warp.  So it has no branches on the tile (rows that
    // are not the group's are added like the others and not stored), and a wait that
    // ran out only makes the later ones return at once.
    auto arrived = [&]() {
      if (!mbar_try_wait(&buf_full[b], bphase)) mbar_wait_inline(&buf_full[b], bphase, abort_flag);
      __syncwarp();
      tc_fence_after();
    };
    for (int u = pair; u < units; u += npairs) {
      const GroupTile t = tile_of<0, TILE>(u, a, table);
      const int rows = t.rows - rank * BM;  // of this CTA
      // this row's scales and those of the 128 x 128 blocks of the weights, two blocks
      // of K ahead
      const float* xp = reinterpret_cast<const float*>(a.xs) +
                        static_cast<int64_t>(t.row0 + (my_row < rows ? rank * BM + my_row : 0)) * a.xs_row;
      const float* wp = static_cast<const float*>(a.ws) +
                        (static_cast<int64_t>(t.e) * a.RTW + min(2 * t.wt + half, a.RTW - 1)) * a.KT;
      float x1 = __ldg(xp), w1 = __ldg(wp), x2 = 0.f, w2 = 0.f;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      // 64 columns at a time; the buffer is given back once the second lot is in
      // registers, before it is added.
      uint32_t r[4][16];
      auto load = [&](uint32_t at) {
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x16(at + 16 * q, r[q]);
      };
      int left = a.KT - 1;  // blocks after this one
      if (left > 0) {
        xp += a.xs_kt;
        x2 = __ldg(xp);
        w2 = __ldg(++wp);
      }
      while (true) {
        arrived();
        load(src + b * TILE);
        const float s = x1 * w1;
        x1 = x2;
        w1 = w2;
        if (left > 1) {
          xp += a.xs_kt;
          x2 = __ldg(xp);
          w2 = __ldg(++wp);
        }
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 64; ++j) add_scaled(acc[j], r[j >> 4][j & 15], s);
        load(src + b * TILE + 64);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(free_bar + static_cast<uint32_t>(b * 8));
        b ^= 1;
        bphase ^= b ^ 1;
#pragma unroll
        for (int j = 0; j < 64; ++j) add_scaled(acc[64 + j], r[j >> 4][j & 15], s);
        if (left-- == 0) break;
      }
      // 32 columns at a time: this thread's row to shared memory, 16-byte pieces
      // swizzled; from there four lanes a row.  (From registers, a lane a row of 32
      // lines an instruction, a tile took 1.9 us.)
      if ((warp & 3) * 32 < rows) {
        const int n0 = t.wt * TILE + half * BM;
        const int row0 = (warp & 3) * 32;
        __nv_bfloat16* out = a.out + static_cast<int64_t>(t.row0 + rank * BM + row0) * a.N + n0;
        const __nv_bfloat16* bias = a.bias != nullptr ? a.bias + t.e * a.bias_stride + n0 : nullptr;
        uint8_t* box = smem + OFF_OUT + ew * OUT_BOX;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (n0 + 32 * q >= a.N) break;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int c = 32 * q + 8 * p;
            uint4 bv = make_uint4(0, 0, 0, 0);
            if (bias != nullptr && n0 + c < a.N) bv = __ldg(reinterpret_cast<const uint4*>(bias + c));
            const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = pack_bf16x2(acc[c + 2 * k] + __uint_as_float(bw[k] << 16),
                                 acc[c + 2 * k + 1] + __uint_as_float(bw[k] & 0xFFFF0000u));
            *reinterpret_cast<uint4*>(box + lane * 64 + (((p ^ (lane >> 1)) & 3) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int r = 8 * p + (lane >> 2), c = 32 * q + 8 * (lane & 3);
            const uint4 v = *reinterpret_cast<const uint4*>(box + r * 64 + ((((lane & 3) ^ (r >> 1)) & 3) << 4));
            if (row0 + r < rows && n0 + c < a.N) *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * a.N + c) = v;
          }
          __syncwarp();
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // Neither CTA leaves while the other may still signal it; the odd CTA's last arrivals
  // on buf_free, which nobody waits for, are ordered by this barrier.
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

}  // namespace

cudaError_t launch_gemm_b128_pair(const GroupedProblem& p, int sms, cudaStream_t stream, const char** msg) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(gemm_b128_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) {
      *msg = "cudaFuncSetAttribute(max dynamic shared memory) failed";
      return e;
    }
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  CUtensorMap mw, mx, mbox;
  if (!grouped_maps(p, BM, &mw, &mx, &mbox)) {
    *msg = "cuTensorMapEncodeTiled rejected an operand of the block-128 product";
    return cudaErrorInvalidValue;
  }
  const GroupedArgs a = grouped_args(p, 2, 1);
  const int64_t units = grouped_max_tiles(p.E, p.R, p.offsets != nullptr, TILE) * a.WT;
  const int64_t pairs = units < sms / 2 ? units : sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_b128_pair_kernel, mw, mx, mbox, a);
  if (e != cudaSuccess) *msg = "block-128 product launch failed";
  return e;
}

cudaError_t take_status_b128_pair(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
}

}  // namespace mx
