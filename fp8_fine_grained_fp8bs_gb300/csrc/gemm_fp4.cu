// 4-bit block-scaled GEMM: E2M1 operands whose block scales the tensor core
// applies, FP32 accumulation in tensor memory, and one float32 scale per row
// of each operand applied in the epilogue:
//
//   D[m][n] = ga[m] gb[n] sum_k (a[m][k] sa[m][k/B]) (b[n][k] sb[n][k/B])
//
// with B = 16 and E4M3 scales (tcgen05.mma.kind::mxf4nvf4, scale_vec::4X) or
// B = 32 and UE8M0 scales (kind::mxf4, scale_vec::2X; no row scales).  One
// MMA takes K = 64: 32 bytes of each operand row, the same bytes as a K = 32
// FP8 MMA, at twice its FLOP rate.
//
// Scales come in the layout tensor memory wants (512-byte blocks of 128 rows
// x 4 groups, see fp4.cu): the producer loads a stage's blocks with TMA next
// to the operand tiles, and the MMA thread copies them into tensor memory
// with tcgen05.cp.32x128b.warpx4 just before the MMAs that read them.  A
// block holds the scales of K = 64 (E4M3x16) or K = 128 (UE8M0x32).  Tensor
// memory keeps one set of scale columns per shared-memory stage, so a set is
// rewritten only after the stage was handed back, which the MMAs that read
// the set do when they complete.
//
// Structure (persistent, warp-specialised): warp 0 producer, warp 1 MMA
// issuer, warps 4-11 epilogue, as in gemm_mx.cu.  Stages are 256 elements of
// K (128 bytes, one swizzle row) deep; the last may be shorter: elements past
// K are zero-filled by TMA and their MMAs are not issued.
//
// Large products run 256x256 tiles on CTA pairs (2-SM MMA).  4096x7168x7168 back
// to back takes 72 us (5850 TFLOP/s) with E4M3 scales; in a run too short for the
// power limit to lower the clock 67 us (6250), and 61 (6920) with UE8M0 ones.
// What bounds it, from variants that leave parts out (4864x4096, four tiles a
// pair, time per stage of four MMAs): the MMAs alone 0.263 us, 545 cycles for
// 512 of tensor work; with the operands' TMA writes, which share shared
// memory's bandwidth with the MMA's reads, 0.30; with the scale copies 0.32; and
// about 10 us a launch outside the stages (start, first loads, accumulators
// handed over between tiles, the last store).  So the rate of the K = 64 MMA is
// the largest part; MMAs of K = 96 were not measured.  A 256-wide tile has one
// accumulator (two would take all of tensor memory and leave none for scales), so
// the next tile's MMAs wait until the epilogue has read it.  Two staging boxes per
// epilogue warp (a stage less in the ring), stores straight from registers and
// prefetching B into L2 were slower.
//
// Grouped products of few rows stream B: 32 experts of [4096][7168], 128 choices,
// 90 us for 520 MB of DRAM traffic (0.85 of the copy bandwidth).
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "block_scale.cuh"
#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "tmap.h"

namespace fp8bs {
namespace {

__device__ int g_gemm_fp4_status;
__device__ __forceinline__ void record_fp4_status(int code) { atomicCAS(&g_gemm_fp4_status, 0, code); }

constexpr int kF4Threads = 384;       // 12 warps
constexpr int kF4EpiWarp0 = 4;
constexpr int kF4EpiThreads = 256;
constexpr uint32_t kF4TmemCols = 512;
constexpr uint32_t kF4RegsControl = 72;     // warps 0-3
constexpr uint32_t kF4RegsEpilogue = 216;   // warps 4-11: 128 accumulators and the store
constexpr uint32_t kF4LaunchRegs = 168;
static_assert(kF4RegsControl * 128 + kF4RegsEpilogue * kF4EpiThreads == kF4LaunchRegs * kF4Threads, "register split");
constexpr int kF4StageK = 256;              // elements of K per stage
constexpr int kF4MmaK = 64;                 // elements of K per MMA
constexpr int kStageMmas = kF4StageK / kF4MmaK;
constexpr int kSfBlockBytes = 512;          // 128 rows x 4 scales

struct F4Params {
  const float* ga;
  const float* gb;
  const int32_t* offsets;
  int64_t M;
  int N;
  int K;
  int nkb;            // stages along K
  int nsb;            // scale blocks along K
  int num_groups;
  int out_bf16;
  uint64_t timeout_ns;
};

template <int kFmt, int BN, bool kGrouped, bool kPair>
struct F4Cfg {
  static constexpr int kABytes = kBlockM * 128;
  static constexpr int kBBytes = (kPair ? BN / 2 : BN) * 128;
  static constexpr int kSfPerStage = kFmt == 0 ? 4 : 2;                 // scale blocks per 128 rows and stage
  static constexpr int kNTiles = (BN + 127) / 128;                      // 128-column scale tiles of B
  static constexpr int kSfABytes = kSfPerStage * kSfBlockBytes;
  static constexpr int kSfBBytes = kNTiles * kSfPerStage * kSfBlockBytes;
  static constexpr int kStageBytes = kABytes + kBBytes + kSfABytes + kSfBBytes;
  static constexpr int kAccBufs = BN == 256 ? 1 : 2;
  static constexpr int kSfCols = kSfPerStage * 4 * (1 + kNTiles);       // tensor memory columns per stage
  static constexpr int kSfBase = kAccBufs * BN;
  static constexpr int kOutBytes = (kF4EpiThreads / 32) * kOutBoxBytes;
  static constexpr int kMaxStages = (static_cast<int>(kF4TmemCols) - kSfBase) / kSfCols;
  static constexpr int kGroupBytes = kGrouped ? 2 * (kMaxGroups + 1) * 4 : 0;
  static constexpr int kTailBytes = (2 * 8 + 2 * 2 + 1) * 8 + 16 + 8 + kGroupBytes;
  static constexpr int kFit = (kSmemBudget - kOutBytes - kTailBytes - 1024) / kStageBytes;
  static constexpr int kStages0 = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kStages = kStages0 < 8 ? kStages0 : 8;
  static_assert(kStages >= 3, "operand ring too shallow");
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kOffA + kStages * kABytes;
  static constexpr int kOffOut = kOffB + kStages * kBBytes;
  static constexpr int kOffSfA = kOffOut + kOutBytes;
  static constexpr int kOffSfB = kOffSfA + kStages * kSfABytes;
  static constexpr int kOffBar = kOffSfB + kStages * kSfBBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffGroups = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffGroups + kGroupBytes + 1024;
  static_assert(kOffOut % 1024 == 0, "staging boxes need 1024-byte alignment for the 128-byte swizzle");
  static_assert(kSmemBytes <= kSmemBudget, "shared memory budget");
};

// Instruction descriptor of the block-scaled 4-bit kinds: B scale id in bits
// 4-5, A and B E2M1 (1 in bits 7-9 and 10-12), both K-major, N >> 3 in bits
// 17-22, scale type in bit 23 (0 E4M3, 1 UE8M0), M >> 4 in bits 24-28, A
// scale id in bits 29-30, K = 64 (bit 31 clear).  The scale ids are zero here.
template <int kFmt>
__host__ __device__ constexpr uint32_t idesc_fp4(int m, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (kFmt == 1 ? 1u << 23 : 0u) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// Four floats of the shared memory of a CTA of the cluster (an address from mapa_shared).
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int kFmt, bool kPair>
__device__ __forceinline__ void mma_fp4(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t tmem_sfa, uint32_t tmem_sfb, uint32_t accumulate) {
#define FP8BS_MMA_FP4(form)                                                                             \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\ttcgen05.mma." form                       \
               " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(tmem_d),                                  \
               "l"(adesc), "l"(bdesc), "r"(idesc), "r"(tmem_sfa), "r"(tmem_sfb), "r"(accumulate)        \
               : "memory")
  if constexpr (kFmt == 0 && kPair) {
    FP8BS_MMA_FP4("cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X");
  } else if constexpr (kFmt == 0) {
    FP8BS_MMA_FP4("cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X");
  } else if constexpr (kPair) {
    FP8BS_MMA_FP4("cta_group::2.kind::mxf4.block_scale.scale_vec::2X");
  } else {
    FP8BS_MMA_FP4("cta_group::1.kind::mxf4.block_scale.scale_vec::2X");
  }
#undef FP8BS_MMA_FP4
}

// Issues one stage's MMAs: copies the stage's scale blocks into its columns
// of tensor memory, then one MMA per 64 elements of K that the stage holds.
// a, b: shared-memory addresses of the tiles; sfa, sfb: of the scale blocks,
// kNTiles tiles of 128 columns of B; sf_col: first tensor memory column of the
// stage's scales; idesc: with scale ids of zero.
template <int kFmt, int kNTiles, bool kPair>
__device__ __forceinline__ void issue_stage(uint32_t dtmem, uint32_t a, uint32_t b, uint32_t sfa, uint32_t sfb,
                                            uint32_t sf_col, uint32_t idesc, int mmas, bool first) {
  constexpr int kBlocks = kFmt == 0 ? 4 : 2;                // scale blocks per 128 rows and stage
  constexpr int kPerBlock = kStageMmas / kBlocks;           // MMAs that read one scale block
  constexpr uint32_t kSfbCol = kBlocks * 4;
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    if (j * kPerBlock < mmas) {
      if (kPair)
        tmem_cp_rows_pair(sf_col + 4 * j, sf_rows_desc(sfa + j * kSfBlockBytes));
      else
        tmem_cp_rows(sf_col + 4 * j, sf_rows_desc(sfa + j * kSfBlockBytes));
#pragma unroll
      for (int h = 0; h < kNTiles; ++h) {
        const uint32_t dst = sf_col + kSfbCol + 4 * (j * kNTiles + h);
        const uint64_t src = sf_rows_desc(sfb + (h * kBlocks + j) * kSfBlockBytes);
        if (kPair)
          tmem_cp_rows_pair(dst, src);
        else
          tmem_cp_rows(dst, src);
      }
    }
  }
  const uint64_t adesc = sw128_kmajor_desc(a), bdesc = sw128_kmajor_desc(b);
#pragma unroll
  for (int k = 0; k < kStageMmas; ++k) {
    if (k < mmas) {
      const int j = k / kPerBlock;
      const uint32_t id = kFmt == 0 ? 0u : 2u * static_cast<uint32_t>(k & 1);
      mma_fp4<kFmt, kPair>(dtmem, adesc + 2 * k, bdesc + 2 * k, idesc | (id << 4) | (id << 29), sf_col + 4 * j,
                           sf_col + kSfbCol + 4 * kNTiles * j, (!first || k > 0) ? 1u : 0u);
    }
  }
}

// Stores a thread's kCols accumulators of row y0 + lane from column x0 on,
// times the row's and the columns' scales: per 128-byte column block the warp
// fills a staging box (128-byte swizzled) and lane 0 stores it with TMA, which
// clips rows and columns past the output; blocks that begin past it are left out.
template <int kFmt, int kCols, bool kBf16>
__device__ __forceinline__ void store_scaled(const float* acc, float ga, const float* gb, uint8_t* box, int lane,
                                             const CUtensorMap* tmD, int x0, int n, int y0) {
  constexpr int kPerChunk = kBf16 ? 8 : 4;
  constexpr int kBoxCols = 8 * kPerChunk;
  static_assert(kCols % kBoxCols == 0, "segment of whole boxes");
#pragma unroll
  for (int b = 0; b < kCols / kBoxCols; ++b) {
    if (x0 + b * kBoxCols < n) {
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      uint8_t* row = box + lane * 128;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float v[kPerChunk];
#pragma unroll
        for (int i = 0; i < kPerChunk; i += 4) {
          const int col = b * kBoxCols + c * kPerChunk + i;
          float4 s = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
          // n is a multiple of 8: four columns are stored whole or not at all
          if (kFmt == 0 && x0 + col < n) s = __ldg(reinterpret_cast<const float4*>(gb + col));
          v[i] = kFmt == 0 ? acc[col] * (ga * s.x) : acc[col];
          v[i + 1] = kFmt == 0 ? acc[col + 1] * (ga * s.y) : acc[col + 1];
          v[i + 2] = kFmt == 0 ? acc[col + 2] * (ga * s.z) : acc[col + 2];
          v[i + 3] = kFmt == 0 ? acc[col + 3] * (ga * s.w) : acc[col + 3];
        }
        uint4 w;
        if constexpr (kBf16)
          w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        else
          w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        *reinterpret_cast<uint4*>(row + ((c ^ (lane & 7)) << 4)) = w;
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(tmD, box, x0 + b * kBoxCols, y0);
        bulk_commit();
      }
    }
  }
}

template <int kFmt, int BN, bool kGrouped, bool kPair>
__global__ void __launch_bounds__(kF4Threads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSfA, const __grid_constant__ CUtensorMap tmSfB,
                    const __grid_constant__ CUtensorMap tmD, const F4Params p) {
  using C = F4Cfg<kFmt, BN, kGrouped, kPair>;
  constexpr int kCols = BN / 2;   // of an epilogue thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem + C::kOffA;
  uint8_t* sB = smem + C::kOffB;
  uint8_t* sSfA = smem + C::kOffSfA;
  uint8_t* sSfB = smem + C::kOffSfB;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [kStages] TMA -> MMA
  uint64_t* empty = full + C::kStages;                              // [kStages] MMA -> TMA
  uint64_t* acc_full = empty + C::kStages;                          // [kAccBufs] tile accumulated
  uint64_t* acc_empty = acc_full + C::kAccBufs;                     // [kAccBufs] accumulator read out
  uint64_t* teardown = acc_empty + C::kAccBufs;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  int* s_off = reinterpret_cast<int*>(smem + C::kOffGroups);
  int* s_cum = s_off + (kMaxGroups + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform, and known to be
  const int lane = threadIdx.x & 31;
  const int ntn = (p.N + BN - 1) / BN;
  const int nst = (p.N + 127) / 128;   // 128-column scale tiles of one B
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const int unit0 = kPair ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int nunits = kPair ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kAccBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], (kPair ? 2 : 1) * kF4EpiThreads / 32);
    }
    mbar_init(&teardown[0], 1);
    fence_barrier_init();
    griddep_wait();  // the group table below may come from the preceding kernel
    int total_mt = 0;
    bool ok = true;
    if (kGrouped) {
      int prev = 0;
      for (int g = 0; g <= p.num_groups; ++g) {
        const int o = p.offsets[g];
        ok = ok && (o >= prev || g == 0) && o >= 0 && (o % kBlockM) == 0 && o <= p.M;
        s_off[g] = o;
        prev = o;
      }
      if (ok) {
        for (int g = 0; g < p.num_groups; ++g) {
          s_cum[g] = total_mt;
          const int mt = (s_off[g + 1] - s_off[g]) / kBlockM;
          total_mt += kPair ? (mt + 1) / 2 : mt;
        }
        s_cum[p.num_groups] = total_mt;
      } else {
        record_fp4_status(kStatusDeviceArg);
        total_mt = 0;
      }
    } else {
      total_mt = static_cast<int>((p.M + kBlockM - 1) / kBlockM);
      if (kPair) total_mt = (total_mt + 1) / 2;
    }
    misc[2] = static_cast<uint32_t>(total_mt * ntn);
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmSfA);
    prefetch_tmap(&tmSfB);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&misc[0], kF4TmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&misc[0], kF4TmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (kPair) cluster_sync();
  griddep_launch_dependents();  // the next kernel may start on the SMs that this one leaves first
  griddep_wait();  // operands, scales and D are touched only after the preceding kernel
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, misc[0], 0);
  const int total_tiles = static_cast<int>(misc[2]);

  if (warp < kF4EpiWarp0) {
    setmaxnreg_dec<kF4RegsControl>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      bool live = true;
      int issued = 0;
      int g = 0;
      for (int t = unit0; t < total_tiles && live; t += nunits) {
        int row0, n0;
        int64_t row_end;
        tile_coords<BN, kPair>(t, ntn, kGrouped, s_off, s_cum, p.num_groups, rank, p.M, row0, n0, g, row_end);
        const int sfa_row = row0 / 128 * p.nsb;
        const int sfb_row = (g * nst + n0 / 128) * p.nsb;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!warp_wait(&empty[stage], phase ^ 1, p.timeout_ns)) { live = false; break; }
          if (elect_one()) {
            uint8_t* da = sA + stage * C::kABytes;
            uint8_t* db = sB + stage * C::kBBytes;
            uint8_t* dsa = sSfA + stage * C::kSfABytes;
            uint8_t* dsb = sSfB + stage * C::kSfBBytes;
            const int sk = kb * C::kSfPerStage;
            if (kPair) {
              if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
              const uint32_t leader_full = mapa_shared(&full[stage], 0);
              tma_load_2d_pair(da, &tmA, leader_full, kb * 128, row0);
              if (kGrouped)
                tma_load_3d_pair(db, &tmB, leader_full, kb * 128, n0 + static_cast<int>(rank) * (BN / 2), g);
              else
                tma_load_2d_pair(db, &tmB, leader_full, kb * 128, n0 + static_cast<int>(rank) * (BN / 2));
              tma_load_2d_pair(dsa, &tmSfA, leader_full, 0, sfa_row + sk);
#pragma unroll
              for (int h = 0; h < C::kNTiles; ++h)
                tma_load_2d_pair(dsb + h * C::kSfABytes, &tmSfB, leader_full, 0, sfb_row + h * p.nsb + sk);
            } else {
              mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
              tma_load_2d(da, &tmA, &full[stage], kb * 128, row0);
              if (kGrouped)
                tma_load_3d(db, &tmB, &full[stage], kb * 128, n0, g);
              else
                tma_load_2d(db, &tmB, &full[stage], kb * 128, n0);
              tma_load_2d(dsa, &tmSfA, &full[stage], 0, sfa_row + sk);
#pragma unroll
              for (int h = 0; h < C::kNTiles; ++h)
                tma_load_2d(dsb + h * C::kSfABytes, &tmSfB, &full[stage], 0, sfb_row + h * p.nsb + sk);
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!live) {
        record_fp4_status(kStatusTimeout);
        for (int s = 0; s < C::kStages && s < issued && (!kPair || rank == 0); ++s) {
          int st = stage - 1 - s;
          uint32_t ph = phase;
          if (st < 0) { st += C::kStages; ph ^= 1; }
          (void)mbar_wait(&full[st], ph, p.timeout_ns);
        }
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      int stage = 0;
      uint32_t phase = 0;
      uint32_t tiles_done = 0;
      bool live = true;
      for (int t = unit0; t < total_tiles && live; t += nunits, ++tiles_done) {
        const uint32_t abuf = tiles_done % C::kAccBufs;
        const uint32_t aphase = (tiles_done / C::kAccBufs) & 1u;
        if (!warp_wait(&acc_empty[abuf], aphase ^ 1u, p.timeout_ns)) { live = false; break; }
        const uint32_t dtmem = tmem_base + abuf * BN;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!warp_wait(&full[stage], phase, p.timeout_ns)) { live = false; break; }
          tc_fence_after_sync();
          const int mmas = min(kStageMmas, (p.K - kb * kF4StageK) / kF4MmaK);
          if (elect_one()) {
            const uint32_t a = smem_u32(sA + stage * C::kABytes), b = smem_u32(sB + stage * C::kBBytes);
            const uint32_t sfa = smem_u32(sSfA + stage * C::kSfABytes), sfb = smem_u32(sSfB + stage * C::kSfBBytes);
            const uint32_t sf_col = tmem_base + C::kSfBase + stage * C::kSfCols;
            constexpr uint32_t kIdesc = idesc_fp4<kFmt>(kPair ? 2 * kBlockM : kBlockM, BN);
            if (mmas == kStageMmas)   // the count known: straight-line issue
              issue_stage<kFmt, C::kNTiles, kPair>(dtmem, a, b, sfa, sfb, sf_col, kIdesc, kStageMmas, kb == 0);
            else
              issue_stage<kFmt, C::kNTiles, kPair>(dtmem, a, b, sfa, sfb, sf_col, kIdesc, mmas, kb == 0);
            if (kPair) {
              mma_commit_pair(&empty[stage], 0x3);
              if (kb + 1 == p.nkb) mma_commit_pair(&acc_full[abuf], 0x3);
            } else {
              mma_commit(&empty[stage]);
              if (kb + 1 == p.nkb) mma_commit(&acc_full[abuf]);
            }
          }
          __syncwarp();
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!live) record_fp4_status(kStatusTimeout);
      // every MMA issued must have completed before TMEM is released
      if (elect_one()) {
        if (kPair)
          mma_commit_pair(&teardown[0], 0x1);
        else
          mma_commit(&teardown[0]);
      }
      __syncwarp();
      (void)mbar_wait(&teardown[0], 0, p.timeout_ns);
    }
  } else {
    setmaxnreg_inc<kF4RegsEpilogue>();
    const int e = warp - kF4EpiWarp0;    // 0..7
    const int quarter = warp & 3;        // TMEM lanes 32*quarter .. +31
    const int colhalf = e >> 2;          // which BN/2 columns this warp stores
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* s_out = smem + C::kOffOut + e * kOutBoxBytes;
    if (lane == 0 && e == 0) prefetch_tmap(&tmD);
    bool live = true;
    uint32_t epi_tiles = 0;
    int g = 0;
    for (int t = unit0; t < total_tiles && live; t += nunits, ++epi_tiles) {
      int row0, n0;
      int64_t row_end;
      tile_coords<BN, kPair>(t, ntn, kGrouped, s_off, s_cum, p.num_groups, rank, p.M, row0, n0, g, row_end);
      const uint32_t abuf = epi_tiles % C::kAccBufs;
      const uint32_t aphase = (epi_tiles / C::kAccBufs) & 1u;
      const int y0 = row0 + quarter * 32;
      const int ncol0 = n0 + colhalf * kCols;
      const bool mine = y0 < row_end && ncol0 < p.N;
      const float ga = kFmt == 0 && mine && y0 + lane < p.M ? __ldg(p.ga + y0 + lane) : 1.0f;
      const float* gb = p.gb + static_cast<int64_t>(g) * p.N + ncol0;
      if (!mbar_wait(&acc_full[abuf], aphase, p.timeout_ns)) {
        live = false;
        break;
      }
      tc_fence_after_sync();
      uint32_t acc[kCols / 32][32];
      const uint32_t taddr = tmem_base + lane_base + abuf * BN + colhalf * kCols;
#pragma unroll
      for (int ch = 0; ch < kCols / 32; ++ch) tmem_ld32(taddr + ch * 32, acc[ch]);
#pragma unroll
      for (int ch = 0; ch < kCols / 32; ++ch) tmem_wait_ld(acc[ch]);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (kPair)
          mbar_arrive_cluster(mapa_shared(&acc_empty[abuf], 0));
        else
          mbar_arrive(&acc_empty[abuf]);
      }
      if (mine) {
        const float* v = reinterpret_cast<const float*>(&acc[0][0]);
        if (p.out_bf16)
          store_scaled<kFmt, kCols, true>(v, ga, gb, s_out, lane, &tmD, ncol0, p.N, y0);
        else
          store_scaled<kFmt, kCols, false>(v, ga, gb, s_out, lane, &tmD, ncol0, p.N, y0);
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    if (!live) record_fp4_status(kStatusTimeout);
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (kPair) cluster_sync();
  if (warp == 1) {
    if (kPair)
      tmem_dealloc_pair(tmem_base, kF4TmemCols);
    else
      tmem_dealloc(tmem_base, kF4TmemCols);
  }
}


// ------------------------------------------------------------ few rows of A
// M <= 128: the product is a stream of B, which takes the MMA's side of 128
// rows: a tile is 128 rows of B (columns of D) times all rows of A (rounded up
// to 16, the MMA's N), so each MMA consumes 4 KB of B whatever M is.  With A on
// the side of 128 rows and 64-column tiles, half the B per MMA and per scale
// copy, one token times [7168][7168] took 9.4 us, and 6.7 with three of four
// MMAs left out.
//
// A cluster of 1, 2, 4 or 8 CTAs shares a tile, each CTA taking a part of K;
// the partial tiles meet in shared memory and every CTA adds up and stores its
// part, rank by rank, so the result does not depend on timing.  Two CTAs share
// an SM while a stage is small.
constexpr int kSkinnyThreads = 192;      // warps 0-3 epilogue, 4 producer, 5 MMA issuer
constexpr uint32_t kSkinnyTmemCols = 256;
constexpr int kSkinnyMaxStages = 6;
constexpr int kSkinnyMinSmem = 78 * 1024;
constexpr int kSkinnyPitch = 128 + 4;    // floats per row of the partial tile

template <int kFmt>
struct SkinnyCfg {
  static constexpr int kBlocks = kFmt == 0 ? 4 : 2;                 // scale blocks per 128 rows and stage
  static constexpr int kWBytes = 128 * 128;                         // 128 rows of B
  static constexpr int kSfBytes = kBlocks * kSfBlockBytes;          // of one operand
  static constexpr int kSfCols = 2 * kBlocks * 4;                   // tensor memory columns per stage
  static int stage_bytes(int rows) { return rows * 128 + kWBytes + 2 * kSfBytes; }
  // accumulators take `rows` columns, rounded up to the 32 that a load reads
  static int max_stages(int rows) {
    return std::min(kSkinnyMaxStages, (static_cast<int>(kSkinnyTmemCols) - (rows + 31) / 32 * 32) / kSfCols);
  }
};

template <int kFmt>
__global__ void __launch_bounds__(kSkinnyThreads, 2)
    gemm_fp4_skinny_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmSfA, const __grid_constant__ CUtensorMap tmSfB,
                           const F4Params p, void* __restrict__ d, int rows, int stages, int split) {
  using S = SkinnyCfg<kFmt>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kSkinnyMaxStages], empty[kSkinnyMaxStages], acc_full, teardown;
  __shared__ uint32_t s_tmem;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int a_bytes = rows * 128;
  uint8_t* sB = smem;                                   // [stages] 128 rows of B
  uint8_t* sA = sB + stages * S::kWBytes;               // [stages] rows of A; a multiple of 16: 1024-byte aligned
  uint8_t* sSfB = sA + stages * a_bytes;
  uint8_t* sSfA = sSfB + stages * S::kSfBytes;
  float* part = reinterpret_cast<float*>(smem);         // the partial tile, once every stage has been read

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = split > 1 ? cluster_ctarank() : 0u;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int ntn = (p.N + 127) / 128;
  const int n0 = tile % ntn * 128, m0 = tile / ntn * 128;
  const int m_rows = min(128, static_cast<int>(p.M) - m0);
  const int kb0 = static_cast<int>(rank) * p.nkb / split, kb1 = static_cast<int>(rank + 1) * p.nkb / split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&teardown, 1);
    fence_barrier_init();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmSfA);
    prefetch_tmap(&tmSfB);
  }
  if (warp == 5) {
    tmem_alloc(&s_tmem, kSkinnyTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  griddep_launch_dependents();  // every CTA holds its tensor memory: the next kernel may start its set-up
  griddep_wait();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, s_tmem, 0);
  bool live = true;

  if (warp == 4) {
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    const int sfb_row = n0 / 128 * p.nsb, sfa_row = m0 / 128 * p.nsb;
    const uint32_t bytes = static_cast<uint32_t>(a_bytes + S::kWBytes + 2 * S::kSfBytes);
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(&empty[stage], phase ^ 1, p.timeout_ns)) { live = false; break; }
      if (elect_one()) {
        const int sk = kb * S::kBlocks;
        mbar_arrive_expect_tx(&full[stage], bytes);
        tma_load_2d(sB + stage * S::kWBytes, &tmB, &full[stage], kb * 128, n0);
        tma_load_2d(sSfB + stage * S::kSfBytes, &tmSfB, &full[stage], 0, sfb_row + sk);
        tma_load_2d(sA + stage * a_bytes, &tmA, &full[stage], kb * 128, m0);
        tma_load_2d(sSfA + stage * S::kSfBytes, &tmSfA, &full[stage], 0, sfa_row + sk);
      }
      __syncwarp();
      ++issued;
      if (++stage == stages) { stage = 0; phase ^= 1; }
    }
    if (!live)
      for (int s = 0; s < stages && s < issued; ++s) {
        int st = stage - 1 - s;
        uint32_t ph = phase;
        if (st < 0) { st += stages; ph ^= 1; }
        (void)mbar_wait(&full[st], ph, p.timeout_ns);
      }
  } else if (warp == 5) {
    int stage = 0;
    uint32_t phase = 0;
    const uint32_t idesc = idesc_fp4<kFmt>(128, rows);
    const uint32_t sf_base = tmem_base + (rows + 31) / 32 * 32;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(&full[stage], phase, p.timeout_ns)) { live = false; break; }
      tc_fence_after_sync();
      const int mmas = min(kStageMmas, (p.K - kb * kF4StageK) / kF4MmaK);
      if (elect_one()) {
        const uint32_t b = smem_u32(sB + stage * S::kWBytes), a = smem_u32(sA + stage * a_bytes);
        const uint32_t sfb = smem_u32(sSfB + stage * S::kSfBytes), sfa = smem_u32(sSfA + stage * S::kSfBytes);
        const uint32_t sf_col = sf_base + stage * S::kSfCols;
        if (mmas == kStageMmas)
          issue_stage<kFmt, 1, false>(tmem_base, b, a, sfb, sfa, sf_col, idesc, kStageMmas, kb == kb0);
        else
          issue_stage<kFmt, 1, false>(tmem_base, b, a, sfb, sfa, sf_col, idesc, mmas, kb == kb0);
        mma_commit(&empty[stage]);
        if (kb + 1 == kb1) mma_commit(&acc_full);
      }
      __syncwarp();
      if (++stage == stages) { stage = 0; phase ^= 1; }
    }
    // every MMA issued must have completed before tensor memory is released
    if (elect_one()) mma_commit(&teardown);
    __syncwarp();
    (void)mbar_wait(&teardown, 0, p.timeout_ns);
  } else if (mbar_wait(&acc_full, 0, p.timeout_ns)) {
    // every MMA of this CTA is done, so no stage is read or written any more;
    // lane = column of D, register = row
    tc_fence_after_sync();
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    for (int r0 = 0; r0 < m_rows; r0 += 32) {
      uint32_t acc[32];
      tmem_ld32(taddr + r0, acc);
      tmem_wait_ld(acc);
      float* out = part + r0 * kSkinnyPitch + warp * 32 + lane;
#pragma unroll
      for (int r = 0; r < 32; ++r)
        if (r0 + r < m_rows) out[r * kSkinnyPitch] = __uint_as_float(acc[r]);
    }
  } else {
    live = false;
  }
  if (!live) record_fp4_status(kStatusTimeout);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (split > 1) cluster_sync();
  // pieces of four columns, dealt over the cluster's threads
  for (int i = static_cast<int>(rank) * kSkinnyThreads + static_cast<int>(threadIdx.x); i < m_rows * 32;
       i += split * kSkinnyThreads) {
    const int row = i >> 5, c = (i & 31) * 4;
    if (n0 + c >= p.N) continue;   // N is a multiple of 8
    const float* src = part + row * kSkinnyPitch + c;
    float4 v;
    if (split == 1) {
      v = *reinterpret_cast<const float4*>(src);
    } else {
      float4 w[8];   // every rank's piece in flight, added in the ranks' order
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < split) w[r] = ld_cluster(mapa_shared(src, static_cast<uint32_t>(r)));
      v = w[0];
#pragma unroll
      for (int r = 1; r < 8; ++r)
        if (r < split) {
          v.x += w[r].x;
          v.y += w[r].y;
          v.z += w[r].z;
          v.w += w[r].w;
        }
    }
    if (kFmt == 0) {
      const float ga = __ldg(p.ga + m0 + row);
      const float4 s = __ldg(reinterpret_cast<const float4*>(p.gb + n0 + c));
      v.x *= ga * s.x;
      v.y *= ga * s.y;
      v.z *= ga * s.z;
      v.w *= ga * s.w;
    }
    const int64_t at = static_cast<int64_t>(m0 + row) * p.N + n0 + c;
    if (p.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(d) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(d) + at) = v;
  }
  __syncwarp();
  if (split > 1) cluster_sync();   // no CTA leaves while another reads its partial tile
  if (warp == 5) tmem_dealloc(tmem_base, kSkinnyTmemCols);
}

// Scale blocks as a 2-D tensor of 512-byte rows; one box is one stage's
// blocks of 128 rows.  Blocks past K belong to the next rows (or are filled
// with zeros past the end) and no MMA reads them.
bool encode_scales(CUtensorMap* map, const uint8_t* base, int64_t blocks, uint32_t box_blocks) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t gdim[2] = {kSfBlockBytes / 4, static_cast<cuuint64_t>(blocks)};
  cuuint64_t gstride[1] = {kSfBlockBytes};
  cuuint32_t box[2] = {kSfBlockBytes / 4, box_blocks};
  cuuint32_t estride[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


F4Params params_of(const Fp4GemmArgs& a, int64_t nsb) {
  F4Params kp;
  kp.ga = a.ga;
  kp.gb = a.gb;
  kp.offsets = a.offsets;
  kp.M = a.M;
  kp.N = static_cast<int>(a.N);
  kp.K = static_cast<int>(a.K);
  kp.nkb = static_cast<int>((a.K + kF4StageK - 1) / kF4StageK);
  kp.nsb = static_cast<int>(nsb);
  kp.num_groups = a.num_groups;
  kp.out_bf16 = a.out_bf16 ? 1 : 0;
  kp.timeout_ns = a.timeout_ns;
  return kp;
}

// Scale blocks along K.
template <int kFmt>
int64_t scale_blocks(int64_t K) {
  constexpr int64_t block_k = kFmt == 0 ? 64 : 128;
  return (K + block_k - 1) / block_k;
}

template <int kFmt, int BN, bool kGrouped, bool kPair>
cudaError_t run_fp4(const Fp4GemmArgs& a, int sm_count, cudaStream_t stream, bool* tmap_failed,
                    bool* reg_check_failed) {
  using C = F4Cfg<kFmt, BN, kGrouped, kPair>;
  auto kern = gemm_fp4_kernel<kFmt, BN, kGrouped, kPair>;
  // once per device: the register count that the split needs, the shared memory allowance
  static std::atomic<int> prepared[kMaxCachedDevices];
  int regs_ok = 0;
  const cudaError_t err = cached_per_device(
      prepared,
      [&](int* v) {
        cudaFuncAttributes attr;
        cudaError_t e = cudaFuncGetAttributes(&attr, kern);
        if (e != cudaSuccess) return e;
        *v = attr.numRegs * kF4Threads >= static_cast<int>(kF4RegsControl * 128 + kF4RegsEpilogue * kF4EpiThreads) ? 2 : 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
      },
      &regs_ok);
  if (err != cudaSuccess) return err;
  if (regs_ok != 2) {
    *reg_check_failed = true;
    return cudaErrorInvalidConfiguration;
  }

  const uint64_t row_bytes = static_cast<uint64_t>(a.K) / 2;
  const int64_t nsb = scale_blocks<kFmt>(a.K);
  const int64_t nst = (a.N + 127) / 128;
  CUtensorMap tmA, tmB, tmSfA, tmSfB, tmD;
  const uint64_t dA[2] = {row_bytes, static_cast<uint64_t>(a.M)};
  const uint64_t sA[1] = {row_bytes};
  bool ok = encode_operand(&tmA, a.a, 2, dA, sA, kBlockM);
  const uint32_t b_rows = kPair ? BN / 2 : BN;
  const uint64_t dB[3] = {row_bytes, static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.num_groups)};
  const uint64_t sB[2] = {row_bytes, row_bytes * static_cast<uint64_t>(a.N)};
  ok = ok && encode_operand(&tmB, a.b, kGrouped ? 3 : 2, dB, sB, b_rows);
  ok = ok && encode_scales(&tmSfA, a.sfa, (a.M + 127) / 128 * nsb, C::kSfPerStage);
  ok = ok && encode_scales(&tmSfB, a.sfb, a.num_groups * nst * nsb, C::kSfPerStage);
  ok = ok && encode_output(&tmD, a.d, a.M, a.N, a.out_bf16, kOutRows);
  if (!ok) {
    *tmap_failed = true;
    return cudaErrorInvalidValue;
  }

  const F4Params kp = params_of(a, nsb);
  const int64_t ntn = (a.N + BN - 1) / BN;
  int64_t mt_bound = kGrouped ? (a.M / kBlockM + a.num_groups) : (a.M + kBlockM - 1) / kBlockM;
  if (kPair) mt_bound = (mt_bound + 1) / 2;
  const int64_t units = mt_bound * ntn;
  static std::atomic<int> cluster_cache[kMaxCachedDevices];  // co-resident clusters, per device
  return launch_persistent<kPair>(kern, units, sm_count, kF4Threads, C::kSmemBytes, stream, cluster_cache, tmA, tmB,
                                  tmSfA, tmSfB, tmD, kp);
}

template <int kFmt>
cudaError_t run_skinny(const Fp4GemmArgs& a, int sm_count, cudaStream_t stream, bool* tmap_failed) {
  using S = SkinnyCfg<kFmt>;
  auto kern = gemm_fp4_skinny_kernel<kFmt>;
  static std::atomic<int> prepared[kMaxCachedDevices];
  int ignored = 0;
  cudaError_t err = cached_per_device(
      prepared,
      [&](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget - 1024);
      },
      &ignored);
  if (err != cudaSuccess) return err;

  const F4Params kp = params_of(a, scale_blocks<kFmt>(a.K));
  const int rows = static_cast<int>((std::min<int64_t>(a.M, 128) + 15) / 16 * 16);
  // Stages of two CTAs on an SM (each also has 1 KB of the system's and 1 KB for
  // alignment), and of K among the CTAs of a cluster: as many CTAs as are
  // resident at once, each with two stages at least.  With K whole, by 2, 4 and 8:
  // M1 N7168 K7168 11.2, 9.2, 8.5, 12.7 us (4 taken); N2048 9.9, 7.1, 5.1, 4.8 (8);
  // M128 N16384 K4096 16.3, 15.4, 22.6, 38.4 (2); M1 N24576 K7168 18.4, 22.8, 25.3,
  // 35.6 (whole); B from DRAM.
  const int stage = S::stage_bytes(rows);
  int stages = std::min(S::max_stages(rows), (kSmemBudget / 2 - 3 * 1024) / stage);
  const int64_t ntn = (a.N + 127) / 128, tiles = (a.M + 127) / 128 * ntn;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= 2 * sm_count && kp.nkb >= split * 2 * 2) split *= 2;
  stages = std::max(2, std::min(stages, (kp.nkb + split - 1) / split));
  const int part = static_cast<int>(std::min<int64_t>(a.M, 128)) * kSkinnyPitch * 4;
  // At least a third of the SM's shared memory, so that never more than two CTAs
  // of 256 tensor memory columns meet on an SM: a third would wait for columns
  // that a CTA holds while it waits, in turn, for a cluster peer elsewhere.
  const int smem = std::max(std::max(stages * stage, part) + 1024, kSkinnyMinSmem);

  const uint64_t row_bytes = static_cast<uint64_t>(a.K) / 2;
  CUtensorMap tmA, tmB, tmSfA, tmSfB;
  const uint64_t dA[2] = {row_bytes, static_cast<uint64_t>(a.M)};
  const uint64_t dB[2] = {row_bytes, static_cast<uint64_t>(a.N)};
  const uint64_t stride[1] = {row_bytes};
  bool ok = encode_operand(&tmA, a.a, 2, dA, stride, static_cast<uint32_t>(rows));
  ok = ok && encode_operand(&tmB, a.b, 2, dB, stride, 128);
  ok = ok && encode_scales(&tmSfA, a.sfa, (a.M + 127) / 128 * kp.nsb, S::kBlocks);
  ok = ok && encode_scales(&tmSfB, a.sfb, ntn * kp.nsb, S::kBlocks);
  if (!ok) {
    *tmap_failed = true;
    return cudaErrorInvalidValue;
  }
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(split);
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), 1, 1);
  cfg.blockDim = dim3(kSkinnyThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = split > 1 ? 2 : 1;
  err = cudaLaunchKernelEx(&cfg, kern, tmA, tmB, tmSfA, tmSfB, kp, a.d, rows, stages, split);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <int kFmt>
cudaError_t pick_fp4(const Fp4GemmArgs& a, int sm_count, cudaStream_t stream, bool* tmap_failed,
                     bool* reg_check_failed) {
  const int64_t mt = (a.M + kBlockM - 1) / kBlockM, nkb = (a.K + kF4StageK - 1) / kF4StageK;
  if (a.offsets != nullptr) {
    // Pairs take the rows of a group two m-tiles at a time: with one m-tile a group
    // their second halves idle (32 experts, N4096 K7168: 4224 rows 90.0 us on single
    // CTAs and 101.9 on pairs, 6144 rows 102.7 and 110.2, 9728 rows 145.3 and 131.7).
    return a.N <= 128 || mt * ((a.N + 255) / 256) < sm_count || a.M <= int64_t(256) * a.num_groups
               ? run_fp4<kFmt, 128, true, false>(a, sm_count, stream, tmap_failed, reg_check_failed)
               : run_fp4<kFmt, 256, true, true>(a, sm_count, stream, tmap_failed, reg_check_failed);
  }
  const int64_t small = mt * ((a.N + 127) / 128), large = (mt + 1) / 2 * ((a.N + 255) / 256);
  // One m-tile; or so few tiles that four CTAs can share each one's K, four stages
  // or more apiece (M256 N4096 K7168: 11.2 us against 13.4 for 128x128 tiles
  // that walk all of K; sharing by two loses, M200 N7168 K7168: 16.3 against 14.5).
  if (a.M <= kBlockM || (small * 4 <= 2 * sm_count && nkb >= 16)) return run_skinny<kFmt>(a, sm_count, stream, tmap_failed);
  // 256x256 tiles of a CTA pair against 128x128 tiles of one CTA by the waves they
  // take: a stage costs 0.40 and 0.36 us, the pairs 1.5 us more to start
  // (M512 N7168 K7168: 17.7 us in one wave of pairs, 24.3 in two of single CTAs;
  // M1000 N4104 K448: 6.8 and 5.7).
  const int64_t waves_small = (small + sm_count - 1) / sm_count, waves_large = (large + sm_count / 2 - 1) / (sm_count / 2);
  return waves_large * nkb * 40 + 150 < waves_small * nkb * 36
             ? run_fp4<kFmt, 256, false, true>(a, sm_count, stream, tmap_failed, reg_check_failed)
             : run_fp4<kFmt, 128, false, false>(a, sm_count, stream, tmap_failed, reg_check_failed);
}

}  // namespace

cudaError_t launch_gemm_fp4(const Fp4GemmArgs& a, int fmt, int sm_count, cudaStream_t stream, bool* tmap_failed,
                            bool* reg_check_failed) {
  *tmap_failed = false;
  *reg_check_failed = false;
  return fmt == 0 ? pick_fp4<0>(a, sm_count, stream, tmap_failed, reg_check_failed)
                  : pick_fp4<1>(a, sm_count, stream, tmap_failed, reg_check_failed);
}

cudaError_t gemm_fp4_take_status(int* status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_gemm_fp4_status, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_gemm_fp4_status, &zero, sizeof(int));
  }
  *status = v;
  return e;
}

}  // namespace fp8bs
