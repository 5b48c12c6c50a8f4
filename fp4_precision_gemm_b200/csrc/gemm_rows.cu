// Grouped blockwise FP8 GEMM for few rows (decoding): C[r, n] = sum over 128-element K chunks of
// sa[kb, r] sb(n, kb) (A[r, kb] . B_e[n, kb]) for the rows r of expert e, promoted to FP32 chunk by
// chunk ("Can you explain the role of FP8 precision in DeepSeek-V3 training", "Increased
// accumulation precision"), exactly as gemm_blockwise_kernel forms it: the same products, chunk
// sums and FP32 operations in the same order.
//
// With a few rows per expert the weights' bytes are the bound.  The 256-row tiles of the large
// kernel would be nearly empty and few, so here the weights take the MMA's 128-row side and
// the tokens its N side: a work unit is 128 weight rows x kRows tokens over all of K.
// One persistent CTA per SM keeps a ring of K chunks (16 KB of weights each) in flight by TMA through
// unit borders; partial sums rotate over four TMEM buffers of kRows columns, and eight warps
// (one weight row and half of the tokens per thread) promote them into registers: a chunk's
// promotion has to fit in the 0.37 us in which HBM delivers a chunk to an SM (four warps: 24
// tokens over 32 experts, K 2048, N 7168 the same, but 64-token units 10% slower).  The row
// blocks of one weight tile are neighbouring units, so the weights come from HBM once and from
// L2 for the other blocks.  1 token x 8 experts, K 7168, N 2048 (117 MB of weights): 29 us
// back to back; 24 tokens x 8 of 32 experts, K 2048, N 7168 (470 MB): 92 us, 5.1 TB/s.
// Every wait is bounded, as in the large kernel.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace fp8q {

using namespace sm100;

namespace {

constexpr int kTileN = 128, kChunk = 128;
constexpr int kBufs = 4, kSlots = 12;
constexpr int kPromoWarps = 8;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kThreads = 11 * 32;
constexpr int kMaxGroups = 256;
constexpr uint64_t kWaitNs = 4000000000ull;
constexpr uint32_t kWBytes = kTileN * kChunk;

// kRows: tokens per unit.
template <int kRows>
struct alignas(1024) Shared {
  static constexpr int kStages = kRows == 32 ? 10 : 8;   // a bit under 200 KB of chunks
  uint8_t w[kStages][kWBytes];
  uint8_t a[kStages][kRows * kChunk];
  float scales[kSlots][kRows + 4];   // a chunk's row scales, then the tile's weight scale
  uint64_t full[kStages], empty[kStages], pfree[kBufs], sfull[kSlots], sempty[kSlots], last;
  int prefix[kMaxGroups + 1], offs[kMaxGroups + 1];   // units before each expert, its rows
  uint32_t tmem;
  volatile int abort_flag;
};

struct Unit {
  int g, m0, mend, n0;
};

template <int kRows>
__device__ __forceinline__ Unit unit_of(int t, const GemmParams& p, const Shared<kRows>& S) {
  int g = 0, past = p.num_groups;   // the last expert with prefix[g] <= t
  while (past - g > 1) {
    const int mid = (g + past) >> 1;
    if (S.prefix[mid] <= t) g = mid;
    else past = mid;
  }
  const int rows = S.offs[g + 1] - S.offs[g], blocks = (rows + kRows - 1) / kRows, local = t - S.prefix[g];
  Unit U;
  U.g = g;
  U.m0 = S.offs[g] + (local % blocks) * kRows;
  U.mend = min(S.offs[g + 1], U.m0 + kRows);
  U.n0 = (local / blocks) * kTileN;
  return U;
}

}  // namespace

template <int kRows, bool DGRAD, bool ACC32>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_few_rows_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap tma_a,
                         const __grid_constant__ CUtensorMap tma_w) {
  constexpr int kStages = Shared<kRows>::kStages;
  constexpr uint32_t kABytes = kRows * kChunk;
  extern __shared__ uint8_t raw[];
  Shared<kRows>& S = *reinterpret_cast<Shared<kRows>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = p.K / kChunk, tiles_n = (p.N + kTileN - 1) / kTileN;
  auto timeout = [&] {
    S.abort_flag = 1;
    atomicExch(p.status, kDevTimeout);
  };

  if (warp == kProducerWarp) {
    // expert offsets, clamped to [previous offset, M] as in the large kernel (recorded, like rows
    // of no expert), and the units before each expert: warp scans over 32 experts at a time
    int prev = 0, units = 0;
    if (lane == 0) S.offs[0] = min(max(p.m_offsets[0], 0), p.M);
    bool bad = lane == 0 && p.m_offsets[0] != 0;
    prev = __shfl_sync(0xFFFFFFFFu, lane == 0 ? S.offs[0] : 0, 0);
    for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
      const int g = g0 + lane;   // expert g ends at offset g + 1
      const int v = g < p.num_groups ? p.m_offsets[g + 1] : 0;
      int end = max(v, prev);
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, end, s);
        if (lane >= s) end = max(end, o);
      }
      end = min(end, p.M);
      int begin = __shfl_up_sync(0xFFFFFFFFu, end, 1);
      if (lane == 0) begin = prev;
      const int n = g < p.num_groups ? (end - begin + kRows - 1) / kRows * tiles_n : 0;
      int incl = n;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, s);
        if (lane >= s) incl += o;
      }
      if (g < p.num_groups) {
        bad |= end != v || (g == p.num_groups - 1 && v != p.M);
        S.offs[g + 1] = end;
        S.prefix[g] = units + incl - n;
      }
      prev = __shfl_sync(0xFFFFFFFFu, end, 31);
      units += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) S.prefix[p.num_groups] = units;
    if (bad && blockIdx.x == 0) atomicExch(p.status, kDevBadArg);
  } else if (warp == kMmaWarp) {
    tmem_alloc(&S.tmem, kBufs * kRows);
    tmem_relinquish();
  } else if (warp == kScaleWarp && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) mbar_init(&S.pfree[i], kPromoWarps);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&S.sfull[i], 32);
      mbar_init(&S.sempty[i], kPromoWarps);
    }
    mbar_init(&S.last, 1);
    S.abort_flag = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int total = S.prefix[p.num_groups];

  if (warp == kProducerWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tma_a);
      tma_prefetch_desc(&tma_w);
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Unit U = unit_of(t, p, S);
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const uint32_t s = it % kStages;
          if (!mbar_wait(&S.empty[s], ((it / kStages) & 1) ^ 1, &S.abort_flag, kWaitNs)) { timeout(); ok = false; break; }
          mbar_arrive_expect_tx(&S.full[s], kWBytes + kABytes);
          tma_load_2d(S.w[s], &tma_w, &S.full[s], kb * kChunk, U.g * p.N + U.n0);
          tma_load_2d(S.a[s], &tma_a, &S.full[s], kb * kChunk, U.m0);
        }
      }
      for (uint32_t j = 0; j < min(it, (uint32_t)kStages); ++j)   // no copy outlives the CTA
        mbar_wait_drain(&S.full[(it - 1 - j) % kStages], ((it - 1 - j) / kStages) & 1, kWaitNs);
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(kRows >> 3) << 17) | ((uint32_t)(kTileN >> 4) << 24);
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const uint32_t s = it % kStages, b = it % kBufs;
          if (!mbar_wait(&S.pfree[b], ((it / kBufs) & 1) ^ 1, &S.abort_flag, kWaitNs) ||
              !mbar_wait(&S.full[s], (it / kStages) & 1, &S.abort_flag, kWaitNs)) { timeout(); ok = false; break; }
          tc_fence_after();
          const uint64_t wdesc = smem_desc(smem_u32(S.w[s]), 16, 1024, 2);
          const uint64_t adesc = smem_desc(smem_u32(S.a[s]), 16, 1024, 2);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f8f6f4(tmem + b * kRows, wdesc + 2 * k, adesc + 2 * k, idesc, k > 0);
          // one commit: the stage is free and the partial sums are in TMEM.  (A promotion warp
          // cannot miss a phase: the stage's next commit waits for TMEM buffers that it frees.)
          mma_commit(&S.empty[s]);
        }
      }
      mma_commit(&S.last);
      mbar_wait_drain(&S.last, 0, kWaitNs);
    }
  } else if (warp == kScaleWarp) {
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Unit U = unit_of(t, p, S);
      const int nb = U.n0 / kTileN;
      const float* sb = p.sb + (int64_t)U.g * (DGRAD ? KB : tiles_n) * p.ld_sb;
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const uint32_t r = it % kSlots;
        int good = 1;
        if (lane == 0 && !(good = mbar_wait(&S.sempty[r], ((it / kSlots) & 1) ^ 1, &S.abort_flag, kWaitNs))) timeout();
        if (!__shfl_sync(0xFFFFFFFFu, good, 0)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < kRows; i += 32) {
          const int m = U.m0 + i + lane;
          const bool in = m < p.M;
          cp_async_4(&S.scales[r][i + lane], p.sa + (in ? (int64_t)kb * p.ld_sa + m : 0), in ? 4u : 0u);
        }
        if (lane == 0)
          cp_async_4(&S.scales[r][kRows], sb + (DGRAD ? (int64_t)kb * p.ld_sb + nb : (int64_t)nb * p.ld_sb + kb), 4u);
        cp_async_arrive_noinc(&S.sfull[r]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < kPromoWarps) {
    // warp: 32 weight rows (TMEM lanes) x half of the tokens
    constexpr int kCols = kRows / 2;
    const int q = warp & 3, col0 = (warp >> 2) * kCols;
    const uint32_t t_lane = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)col0;
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Unit U = unit_of(t, p, S);
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const uint32_t r = it % kSlots, s = it % kStages, b = it % kBufs;
        if (!mbar_wait(&S.sfull[r], (it / kSlots) & 1, &S.abort_flag, kWaitNs) ||
            !mbar_wait(&S.empty[s], (it / kStages) & 1, &S.abort_flag, kWaitNs)) { timeout(); ok = false; break; }
        tc_fence_after();
        uint32_t v[kCols / 16][16];
#pragma unroll
        for (int h = 0; h < kCols / 16; ++h) tmem_ld_32x32b_x16(t_lane + b * kRows + h * 16, v[h]);
        const float2 sb2 = make_float2(S.scales[r][kRows], S.scales[r][kRows]);
#pragma unroll
        for (int h = 0; h < kCols / 16; ++h) tmem_ld_wait(v[h]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&S.pfree[b]);
#pragma unroll
        for (int h = 0; h < kCols / 16; ++h)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 sa = ld_shared_f4(&S.scales[r][col0 + h * 16 + i]);
            const int a = h * 8 + i / 2;
            acc[a] = __ffma2_rn(make_float2(__uint_as_float(v[h][i]), __uint_as_float(v[h][i + 1])),
                                __fmul2_rn(make_float2(sa.x, sa.y), sb2), acc[a]);
            acc[a + 1] = __ffma2_rn(make_float2(__uint_as_float(v[h][i + 2]), __uint_as_float(v[h][i + 3])),
                                    __fmul2_rn(make_float2(sa.z, sa.w), sb2), acc[a + 1]);
          }
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&S.sempty[r]);
      }
      if (!ok) break;
      // thread = column n of C: a warp's 32 neighbouring values of one row per store
      const int n = U.n0 + q * 32 + lane;
      if (n < p.N) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          if (U.m0 + col0 + i < U.mend) {
            const float x = (i & 1) ? acc[i / 2].y : acc[i / 2].x;
            const int64_t at = (int64_t)(U.m0 + col0 + i) * p.ldc + n;
            if constexpr (ACC32) p.c32[at] = __fadd_rn(p.c32[at], x);
            else reinterpret_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(x);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kBufs * kRows);
  }
}

template <int kRows, bool DGRAD, bool ACC32>
static cudaError_t launch(const GemmParams& p, const CUtensorMap& a, const CUtensorMap& w, int num_sms, cudaStream_t s) {
  auto kern = gemm_few_rows_kernel<kRows, DGRAD, ACC32>;
  const int smem = (int)sizeof(Shared<kRows>) + 1024;
  static_assert(sizeof(Shared<kRows>) + 1024 <= 227 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // at most this many units, whatever the offsets hold
  const int64_t blocks = (int64_t)p.M / kRows + (p.num_groups < p.M ? p.num_groups : p.M);
  const int64_t units = blocks * ((p.N + kTileN - 1) / kTileN);
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  kern<<<(int)(units < num_sms ? units : num_sms), kThreads, smem, s>>>(p, a, w);
  return cudaGetLastError();
}

// Which kernel, by waves of work units (the offsets are on the device, so the experts' row blocks
// are estimated: half a block of padding each, and at least one block).  A wave of this kernel
// (128 weight rows x 64 tokens per SM) costs about 8/13 of one of the large kernel (256 x 256
// per SM pair) at the same K.  Measured, back to back, this kernel against the large one, K x N:
//   32 experts:  8 rows 29 against 38 us (7168 x 2048), 1024 rows 109 / 145, 2048 rows 125 / 145,
//                4096 rows 202 / 150;  2048 x 7168: 31 / 46, 116 / 153, 136 / 150, 213 / 155
//   8 experts:   256 rows 31 / 38, 512 rows 49 / 38;  2048 x 7168: 35 / 46, 41 / 45, 1024 rows 61 / 47
//   64 experts:  4092 rows 230 / 285;  2048 x 7168: 250 / 326
// 32 tokens per unit instead of 64 win where nearly every expert has fewer (64 rows over 32
// experts 76 against 81 us, 8 rows 29 / 30) and lose beyond (1020 rows over 64: 242 / 194).
int gemm_few_rows_tile(int64_t M, int64_t N, int groups, int num_sms) {
  const int64_t hit = groups < M ? groups : M;
  auto waves = [&](int64_t rows, int64_t cols, int64_t slots) {
    const int64_t blocks = M / rows + hit / 2;
    return ((blocks > hit ? blocks : hit) * ((N + cols - 1) / cols) + slots - 1) / slots;
  };
  if (waves(64, 128, num_sms) * 8 > waves(256, 256, num_sms / 2) * 13) return 0;
  return M <= 8 * (int64_t)groups ? 32 : 64;
}

cudaError_t launch_gemm_few_rows(const GemmParams& p, const CUtensorMap& tma_a, const CUtensorMap& tma_w, int num_sms,
                                 cudaStream_t s) {
#define FP8Q_FEW(R, D, A) \
  if (gemm_few_rows_tile(p.M, p.N, p.num_groups, num_sms) == R && (p.layout == 1) == D && (p.c32 != nullptr) == A) \
    return launch<R, D, A>(p, tma_a, tma_w, num_sms, s);
  FP8Q_FEW(32, false, false) FP8Q_FEW(32, false, true) FP8Q_FEW(32, true, false) FP8Q_FEW(32, true, true)
  FP8Q_FEW(64, false, false) FP8Q_FEW(64, false, true) FP8Q_FEW(64, true, false) FP8Q_FEW(64, true, true)
#undef FP8Q_FEW
  return cudaErrorInvalidValue;
}

}  // namespace fp8q
