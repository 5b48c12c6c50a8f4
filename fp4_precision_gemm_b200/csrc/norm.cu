// The norms on both sides of a block's residual connection, fused with its gate and residual
// scale, and their gradients.  With rms(v) = 1 / sqrt(mean(v^2) + eps) over a row of C columns:
//   forward    z = y rms(y) w_post  (or y),   h' = alpha h + gate z,   n = h' rms(h') w_pre,
//              h' stored in the residual's type, n in BF16 and / or as 1x128 E4M3 codes.
//   backward   with xh = h' rms(h'), a = dn w_pre:  d = dh' + rms(h') (a - xh mean(a xh)),
//              dh = alpha d,  dw_pre = sum over rows of dn xh;  with yh = y rms(y) (or y) and
//              S = sum over rows of d yh:  dgate = w_post S,  dw_post = gate S,  and with
//              b = d gate w_post:  dy = rms(y) (b - yh mean(b yh))  (or d gate).
//
// Bound by bytes: every row is read once and written once.  Persistent CTAs take whole rows;
// a thread owns the same NV groups of 8 columns of every row, 16 neighbouring lanes one 128-column
// quantization tile.  Rows arrive in shared memory by bulk copies a few rows ahead (one thread
// issues them), so the loads of the next rows are in flight through both row sums of the
// current one.  All arithmetic and sums are FP32; stored values are rounded once.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace fp8q {

using namespace sm100;

namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxStages = 4;
constexpr uint64_t kNormWaitNs = 4000000000ull;

__device__ __forceinline__ uint32_t pack_bf16_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 consecutive values (16-byte aligned: BF16 one vector, FP32 two).
template <bool F32>
__device__ __forceinline__ void get8(const uint8_t* row, int col, float (&x)[8]) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4*>(row + (size_t)col * 4);
    const float4 b = *reinterpret_cast<const float4*>(row + (size_t)col * 4 + 16);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(row + (size_t)col * 2);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(w[k]), x[2 * k + 1] = bf16_hi(w[k]);
  }
}

template <bool F32>
__device__ __forceinline__ void put8(uint8_t* row, int col, const float (&x)[8]) {
  if constexpr (F32) {
    *reinterpret_cast<float4*>(row + (size_t)col * 4) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(row + (size_t)col * 4 + 16) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(row + (size_t)col * 2) =
        make_uint4(pack_bf16_rn(x[0], x[1]), pack_bf16_rn(x[2], x[3]), pack_bf16_rn(x[4], x[5]), pack_bf16_rn(x[6], x[7]));
  }
}

// Sum over the CTA in a fixed order (lanes, then warps), the same in every thread.  `sh` (zero
// where there is no warp) must not be the buffer of the previous sum; `ok` becomes whether
// every thread's was set.
__device__ __forceinline__ float row_sum(float v, float* sh, int& ok) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  ok = __syncthreads_and(ok);
  const float4* q = reinterpret_cast<const float4*>(sh);
  const float4 a = q[0], b = q[1], c = q[2], d = q[3];
  return (((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w))) +
         (((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w)));
}

struct NormShared {
  alignas(16) float sums[2][kMaxWarps];
  uint64_t full[2 * kMaxStages];
  volatile int abort_flag;   // set by the first thread whose wait runs out: the others stop waiting
};

// The thread's columns of the weights, in FP32: w_pre, and gate * w_post (1 for the missing
// ones).  Kept in registers over all rows where they fit (KEEP), else read again for every row.
template <int NV, bool W32, bool KEEP>
struct Weights {
  float pre[KEEP ? NV : 1][8], mid[KEEP ? NV : 1][8];

  static __device__ __forceinline__ void load_pre(const NormParams& p, int col, float (&w)[8]) {
    get8<W32>(static_cast<const uint8_t*>(p.w_pre), col, w);
  }
  static __device__ __forceinline__ void load_mid(const NormParams& p, int col, float (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 1.0f;
    if (p.w_post != nullptr) get8<W32>(static_cast<const uint8_t*>(p.w_post), col, w);
    if (p.gate != nullptr) {
      float g[8];
      get8<W32>(static_cast<const uint8_t*>(p.gate), col, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] *= g[k];
    }
  }
  __device__ __forceinline__ void init(const NormParams& p, int tid, int T) {
    if constexpr (KEEP) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int col = (v * T + tid) * 8;
        if (col < p.cols) {
          load_pre(p, col, pre[v]);
          load_mid(p, col, mid[v]);
        }
      }
    }
  }
  __device__ __forceinline__ void get_pre(const NormParams& p, int v, int col, float (&w)[8]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = pre[v][k];
    } else {
      load_pre(p, col, w);
    }
  }
  __device__ __forceinline__ void get_mid(const NormParams& p, int v, int col, float (&w)[8]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = mid[v][k];
    } else {
      load_mid(p, col, w);
    }
  }
};

__device__ __forceinline__ float rms_factor(float sum, float inv_cols, float eps) {
  return __frsqrt_rn(fmaf(sum, inv_cols, eps));
}

// Sum of the thread's NV parts (one chain of dependent additions per part keeps them short).
template <int NV>
__device__ __forceinline__ float add_parts(const float (&v)[NV]) {
  if constexpr (NV == 4) return (v[0] + v[1]) + (v[2] + v[3]);
  else if constexpr (NV == 2) return v[0] + v[1];
  else return v[0];
}

}  // namespace

// A stage holds one row of y, then one of h.
template <int NV, bool H32, bool W32>
__global__ void __launch_bounds__(512) norm_forward_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ NormShared sh;
  const int tid = threadIdx.x, T = blockDim.x, C = p.cols;
  const uint32_t ybytes = (uint32_t)C * 2, hbytes = (uint32_t)C * (H32 ? 4 : 2), stage = ybytes + hbytes;
  const bool post = p.w_post != nullptr;
  if (tid < 2 * kMaxWarps) sh.sums[0][tid] = 0.0f;
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&sh.full[s], 1);
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  auto load = [&](int64_t row, int s) {   // thread 0
    mbar_arrive_expect_tx(&sh.full[s], stage);
    bulk_load(ring + s * stage, static_cast<const uint8_t*>(p.y) + row * p.ld_y * 2, ybytes, &sh.full[s]);
    bulk_load(ring + s * stage + ybytes, static_cast<const uint8_t*>(p.h) + row * p.ld_h * (H32 ? 4 : 2), hbytes,
              &sh.full[s]);
  };
  const int64_t step = gridDim.x;
  uint32_t issued = 0;
  if (tid == 0)
    for (; issued < (uint32_t)p.stages; ++issued) {
      const int64_t row = blockIdx.x + issued * step;
      if (row >= p.rows) break;
      load(row, issued);
    }
  Weights<NV, W32, true> W;
  W.init(p, tid, T);
  const float inv_c = 1.0f / (float)C;
  uint32_t it = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += step, ++it) {
    const int s = it % p.stages;
    int ok = mbar_wait(&sh.full[s], (it / p.stages) & 1, &sh.abort_flag, kNormWaitNs);
    if (!ok) sh.abort_flag = 1;
    const uint8_t* ys = ring + s * stage;
    const uint8_t* hs = ys + ybytes;
    float rq = 1.0f;
    if (post) {
      float ss[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int col = (v * T + tid) * 8;
        ss[v] = 0.0f;
        if (col < C) {
          float y[8];
          get8<false>(ys, col, y);
#pragma unroll
          for (int k = 0; k < 8; ++k) ss[v] = fmaf(y[k], y[k], ss[v]);
        }
      }
      rq = rms_factor(row_sum(add_parts(ss), sh.sums[0], ok), inv_c, p.eps);
    }
    float x[NV][8], ss[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (v * T + tid) * 8;
      ss[v] = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[v][k] = 0.0f;
      if (col < C) {
        float y[8], h[8], w[8];
        get8<false>(ys, col, y);
        get8<H32>(hs, col, h);
        W.get_mid(p, v, col, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[v][k] = fmaf(p.alpha, h[k], y[k] * rq * w[k]);
          ss[v] = fmaf(x[v][k], x[v][k], ss[v]);
        }
      }
    }
    const float rp = rms_factor(row_sum(add_parts(ss), sh.sums[post ? 1 : it & 1], ok), inv_c, p.eps);
    if (!ok) break;
    // every thread has read the stage
    if (tid == 0 && row + p.stages * step < p.rows) {
      load(row + p.stages * step, s);
      ++issued;
    }
    uint8_t* hout = static_cast<uint8_t*>(p.h_out) + row * p.ld_h_out * (H32 ? 4 : 2);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (v * T + tid) * 8;
      const bool in = col < C;
      float n[8];
      if (in) {
        float w[8];
        put8<H32>(hout, col, x[v]);
        W.get_pre(p, v, col, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k] = x[v][k] * rp * w[k];
        if (p.n_out != nullptr) put8<false>(static_cast<uint8_t*>(p.n_out) + row * p.ld_n * 2, col, n);
      }
      if (p.q_row != nullptr) {   // C % 128 == 0: a tile's 16 lanes are in or out together
        float am = 0.0f;
        if (in) {
#pragma unroll
          for (int k = 0; k < 8; ++k) am = fmaxf(am, fabsf(n[k]));
        }
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, m));
        if (in) {
          const float sf = e4m3_sf(am);
          uint32_t c[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) c[k] = cvt_e4m3x2(n[2 * k] * sf, n[2 * k + 1] * sf);
          *reinterpret_cast<uint2*>(p.q_row + row * C + col) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
          if ((tid & 15) == 0) p.s_row[(int64_t)(col >> 7) * p.ld_s_row + row] = __frcp_rn(sf);
        }
      }
    }
    if (tid == 0) {
      if (p.rstd_pre != nullptr) p.rstd_pre[row] = rp;
      if (post && p.rstd_post != nullptr) p.rstd_post[row] = rq;
    }
  }
  if (tid == 0) {
    if (it < issued) {   // gave up: report, and leave no copy in flight
      atomicExch(p.status, kDevTimeout);
      for (uint32_t j = it; j < issued; ++j) mbar_wait_drain(&sh.full[j % p.stages], (j / p.stages) & 1, kNormWaitNs);
    }
  }
}

// A stage holds one row of dn, h', dh' (group A, free after the second row sum) and y (group Y,
// read until the row's end).  Column sums stay in registers over all of the CTA's rows and
// leave as one partial row per CTA: partial[cta][0][C] = sum dn xh, [cta][1][C] = sum d yh.
template <int NV, bool H32, bool W32>
__global__ void __launch_bounds__(512) norm_backward_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ NormShared sh;
  const int tid = threadIdx.x, T = blockDim.x, C = p.cols, S = p.stages;
  constexpr int HB = H32 ? 4 : 2;
  const uint32_t nbytes = (uint32_t)C * 2, hbytes = (uint32_t)C * HB, stage = 2 * nbytes + 2 * hbytes;
  const bool post = p.w_post != nullptr;
  uint64_t* full_a = sh.full;
  uint64_t* full_y = sh.full + kMaxStages;
  if (tid < 2 * kMaxWarps) sh.sums[0][tid] = 0.0f;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_a[s], 1);
      mbar_init(&full_y[s], 1);
    }
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int64_t step = gridDim.x, mine = (p.rows - blockIdx.x + step - 1) / step;   // rows of this CTA
  auto load_a = [&](int64_t j) {   // thread 0; j-th row of this CTA
    if (j >= mine) return;
    const int s = (int)(j % S);
    const int64_t row = blockIdx.x + j * step;
    uint8_t* dst = ring + s * stage;
    mbar_arrive_expect_tx(&full_a[s], nbytes + 2 * hbytes);
    bulk_load(dst, static_cast<const uint8_t*>(p.dn) + row * p.ld_dn * 2, nbytes, &full_a[s]);
    bulk_load(dst + nbytes, static_cast<const uint8_t*>(p.h) + row * p.ld_h * HB, hbytes, &full_a[s]);
    bulk_load(dst + nbytes + hbytes, static_cast<const uint8_t*>(p.dh_in) + row * p.ld_dh_in * HB, hbytes, &full_a[s]);
  };
  auto load_y = [&](int64_t j) {
    if (j >= mine) return;
    const int s = (int)(j % S);
    const int64_t row = blockIdx.x + j * step;
    mbar_arrive_expect_tx(&full_y[s], nbytes);
    bulk_load(ring + s * stage + nbytes + 2 * hbytes, static_cast<const uint8_t*>(p.y) + row * p.ld_y * 2, nbytes,
              &full_y[s]);
  };
  if (tid == 0)
    for (int j = 0; j < S; ++j) {
      load_a(j);
      load_y(j);
    }
  float acc_pre[NV][8], acc_s[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc_pre[v][k] = acc_s[v][k] = 0.0f;
  Weights<NV, W32, (NV <= 2)> W;
  W.init(p, tid, T);
  const float inv_c = 1.0f / (float)C;
  int64_t j = 0;
  int ok = 1;
  for (; j < mine; ++j) {
    const int64_t row = blockIdx.x + j * step;
    const int s = (int)(j % S);
    const uint32_t ph = (uint32_t)(j / S) & 1;
    ok = mbar_wait(&full_a[s], ph, &sh.abort_flag, kNormWaitNs) && mbar_wait(&full_y[s], ph, &sh.abort_flag, kNormWaitNs);
    if (!ok) sh.abort_flag = 1;
    const uint8_t* dns = ring + s * stage;
    const uint8_t* hs = dns + nbytes;
    const uint8_t* dhs = hs + hbytes;
    const uint8_t* ys = dhs + hbytes;
    const float rp = p.rstd_pre[row], rq = post ? p.rstd_post[row] : 1.0f;
    float part[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (v * T + tid) * 8;
      part[v] = 0.0f;
      if (col < C) {
        float dn[8], h[8], w[8];
        get8<false>(dns, col, dn);
        get8<H32>(hs, col, h);
        W.get_pre(p, v, col, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float t = dn[k] * (h[k] * rp);
          acc_pre[v][k] += t;
          part[v] = fmaf(t, w[k], part[v]);
        }
      }
    }
    const float c1 = row_sum(add_parts(part), sh.sums[post ? 0 : j & 1], ok) * inv_c;
    if (!ok) break;
    // every thread has left row j - 1: its stage's remaining parts may be refilled
    if (tid == 0 && j > 0 && S > 1) {
      if (!post) load_a(j - 1 + S);
      load_y(j - 1 + S);
    }
    float d[NV][8];
    uint8_t* dh = static_cast<uint8_t*>(p.dh) + row * p.ld_dh * HB;
    uint8_t* dy = static_cast<uint8_t*>(p.dy) + row * p.ld_dy * 2;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (v * T + tid) * 8;
      part[v] = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) d[v][k] = 0.0f;
      if (col < C) {
        float dn[8], h[8], g[8], w[8], t[8];
        get8<false>(dns, col, dn);
        get8<H32>(hs, col, h);
        get8<H32>(dhs, col, g);
        W.get_pre(p, v, col, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          d[v][k] = fmaf(rp, dn[k] * w[k] - h[k] * rp * c1, g[k]);
          t[k] = d[v][k] * p.alpha;
        }
        put8<H32>(dh, col, t);
        float y[8];
        get8<false>(ys, col, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc_s[v][k] = fmaf(d[v][k], y[k] * rq, acc_s[v][k]);
        W.get_mid(p, v, col, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          d[v][k] *= w[k];
          part[v] = fmaf(d[v][k], y[k] * rq, part[v]);
        }
        if (!post) put8<false>(dy, col, d[v]);
      }
    }
    if (post) {
      const float c2 = row_sum(add_parts(part), sh.sums[1], ok) * inv_c;
      if (tid == 0) load_a(j + S);   // dn, h', dh' of row j have been read by every thread
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int col = (v * T + tid) * 8;
        if (col < C) {
          float y[8];
          get8<false>(ys, col, y);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = rq * (d[v][k] - y[k] * rq * c2);
          put8<false>(dy, col, y);
        }
      }
    }
    if (S == 1) {   // wide rows: the only stage is refilled when every thread has left this row
      __syncthreads();
      if (tid == 0) {
        if (!post) load_a(j + 1);
        load_y(j + 1);
      }
    }
  }
  if (!ok) {   // gave up at row j: report, and leave no copy in flight
    if (tid == 0) {
      atomicExch(p.status, kDevTimeout);
      const int late = j > 0 && S > 1;   // the parts of row j - 1 + S are not on their way yet
      for (int64_t i = j; i < j + S && i < mine; ++i) {
        const uint32_t ph = (uint32_t)(i / S) & 1;
        if (i < j + S - (post ? 0 : late)) mbar_wait_drain(&full_a[i % S], ph, kNormWaitNs);
        if (i < j + S - late) mbar_wait_drain(&full_y[i % S], ph, kNormWaitNs);
      }
    }
    return;
  }
  float* part = p.partials + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = (v * T + tid) * 8;
    if (col < C) {
      put8<true>(reinterpret_cast<uint8_t*>(part), col, acc_pre[v]);
      put8<true>(reinterpret_cast<uint8_t*>(part + C), col, acc_s[v]);
    }
  }
}

// Column sums of the CTAs' partials, in CTA order within each of 8 interleaved strands and then
// over the strands: dw_pre, and dw_post / dgate from the sum S of d yh.
template <bool W32>
__global__ void __launch_bounds__(256) norm_columns_kernel(const __grid_constant__ NormParams p, int ctas) {
  __shared__ float sh[2][8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int C = p.cols, col = blockIdx.x * 32 + tx;
  float a = 0.0f, b = 0.0f;
  if (col < C)
#pragma unroll 8
    for (int k = ty; k < ctas; k += 8) {
      const float* part = p.partials + (int64_t)k * 2 * C + col;
      a += part[0];
      b += part[C];
    }
  sh[0][ty][tx] = a;
  sh[1][ty][tx] = b;
  __syncthreads();
  if (ty != 0 || col >= C) return;
  for (int k = 1; k < 8; ++k) {
    a += sh[0][k][tx];
    b += sh[1][k][tx];
  }
  auto weight = [&](const void* w) {
    return w == nullptr ? 1.0f : W32 ? static_cast<const float*>(w)[col]
                                     : bf16_bits_to_float(static_cast<const uint16_t*>(w)[col]);
  };
  p.dw_pre[col] = a;
  if (p.dw_post != nullptr) p.dw_post[col] = b * weight(p.gate);
  if (p.dgate != nullptr) p.dgate[col] = b * weight(p.w_post);
}

namespace {

constexpr int kRingBytes = 220 * 1024;   // shared memory of an SM's rows; no launch takes more

struct NormShape {
  int nv, threads, stages, smem, grid;
};

// Threads own nv groups of 8 columns (512 threads at most): four in the forward kernel (`wide`),
// so that an SM holds several CTAs whose row sums and barriers hide behind one another (8192 x
// 7168, FP32 residual: 115 us, 5.6 TB/s), as few as possible in the backward kernel, whose
// column sums and weights fill the registers (190 us, 5.6 TB/s).  It goes by the columns alone, so
// that a row's result does not depend on how many rows come with it: 4 rows of 7168 take 11 us
// instead of 9 with twice the threads, but sums over the threads in an order of the columns alone
// would cost the large case 5%.  Up to 4 rows are staged per CTA, as many as its share of shared
// memory takes.
NormShape norm_shape(int64_t rows, int cols, int row_bytes, int num_sms, bool wide) {
  NormShape s;
  const int vecs = (cols + 7) / 8;
  s.nv = wide ? 4 : vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
  s.threads = ((vecs + s.nv - 1) / s.nv + 31) / 32 * 32;
  int ctas = 512 / s.threads;
  if (ctas > kRingBytes / (row_bytes + 1024)) ctas = kRingBytes / (row_bytes + 1024);
  if (ctas < 1) ctas = 1;
  s.stages = (kRingBytes / ctas - 1024) / row_bytes;
  if (s.stages > kMaxStages) s.stages = kMaxStages;
  if (s.stages < 1) s.stages = 1;
  s.smem = s.stages * row_bytes;
  const int64_t g = (int64_t)ctas * num_sms;
  s.grid = (int)(rows < g ? rows : g);
  return s;
}

// The limit belongs to the kernel, which calls of other widths share: always the same value, so that another
// thread's call between these two lines changes nothing.
template <class K>
cudaError_t launch_rows(K kern, const NormShape& s, const NormParams& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  kern<<<s.grid, s.threads, s.smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

int norm_backward_ctas(int64_t rows, int cols, bool h32, int num_sms) {
  return norm_shape(rows, cols, cols * (h32 ? 12 : 8), num_sms, false).grid;
}

#define FP8Q_NORM(KERNEL, N, H, W) \
  if (s.nv == N && h32 == H && w32 == W) return launch_rows(KERNEL<N, H, W>, s, q, st);
#define FP8Q_NORMS(KERNEL, N)                                          \
  FP8Q_NORM(KERNEL, N, false, false) FP8Q_NORM(KERNEL, N, false, true) \
  FP8Q_NORM(KERNEL, N, true, false) FP8Q_NORM(KERNEL, N, true, true)

cudaError_t launch_norm_forward(const NormParams& p, bool h32, bool w32, int num_sms, cudaStream_t st) {
  const NormShape s = norm_shape(p.rows, p.cols, p.cols * (h32 ? 6 : 4), num_sms, true);
  NormParams q = p;
  q.stages = s.stages;
  FP8Q_NORMS(norm_forward_kernel, 4)
  return cudaErrorInvalidValue;
}

static cudaError_t launch_norm_backward_rows(const NormParams& p, bool h32, bool w32, const NormShape& s, cudaStream_t st) {
  NormParams q = p;
  q.stages = s.stages;
  FP8Q_NORMS(norm_backward_kernel, 1)
  FP8Q_NORMS(norm_backward_kernel, 2)
  FP8Q_NORMS(norm_backward_kernel, 4)
  return cudaErrorInvalidValue;
}
#undef FP8Q_NORMS
#undef FP8Q_NORM

cudaError_t launch_norm_backward(const NormParams& p, bool h32, bool w32, int num_sms, cudaStream_t st) {
  int ctas = 0;
  if (p.rows > 0) {
    const NormShape s = norm_shape(p.rows, p.cols, p.cols * (h32 ? 12 : 8), num_sms, false);
    const cudaError_t e = launch_norm_backward_rows(p, h32, w32, s, st);
    if (e != cudaSuccess) return e;
    ctas = s.grid;
  }
  const int grid = (p.cols + 31) / 32;
  if (w32) norm_columns_kernel<true><<<grid, 256, 0, st>>>(p, ctas);
  else norm_columns_kernel<false><<<grid, 256, 0, st>>>(p, ctas);
  return cudaGetLastError();
}

}  // namespace fp8q
