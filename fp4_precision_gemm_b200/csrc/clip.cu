// Global gradient norm over many tensors, and their clipped copies:
//   norm = sqrt(sum over all tensors of g^2),  coef = min(1, max_norm / (norm + eps)),
//   out = coef * g (rounded once).
//
// Bound by bytes: every gradient is read for the norm, read again for the scaling and written.
// The tensors are cut into 16 KB chunks that start at whole 128-byte lines of memory; the chunks of
// all tensors are one list over which persistent CTAs stride, so a launch's ramp and tail are paid
// once and small tensors share a wave.  The next chunk's loads are in flight under the current
// one's arithmetic.  The scaling pass walks the list from its end: what the norm pass read last is
// still in L2; its stores are marked as not to be kept there.
//
// Two launches, no atomics: each CTA of the norm pass writes one FP64 partial, and every CTA of
// the scaling pass adds all partials in the same order, so results do not change from run to run.
// Squares: eight values at a time in FP32 (their sum is then off by at most a few 2^-24 of
// itself, far below what is asked of a norm), added up in FP64.  A group whose FP32 sum could
// have overflowed or lost squares to underflow is squared again in FP64, so gradients of any
// finite size give a finite, exact norm.
#include <cfloat>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"

namespace fp8q {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                                    // 16-byte vectors per thread and chunk
constexpr int kChunkBytes = kThreads * kVecs * 16;
constexpr int kLine = 128;                                  // chunks start at whole cache lines

// One chunk: 16-byte vectors from a whole line on, covering elements [e0, e0 + chunk) of tensor i;
// elements outside [0, numel) belong to nobody (the tensor's unaligned head and its tail).
struct Chunk {
  int i, esize;
  int64_t e0, n;
  const uint8_t* g;   // address of element e0 (a whole line's)
};

// The tensor of chunk c.
template <int MAX>
__device__ __forceinline__ int tensor_of(const ClipTensors<MAX>& P, int c) {
  int lo = 0, hi = P.n;                 // chunk_begin[lo] <= c < chunk_begin[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (P.chunk_begin[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Chunk c, its tensor found from `lo`, that of the CTA's chunk before it.
template <int MAX>
__device__ __forceinline__ Chunk chunk_of(const ClipTensors<MAX>& P, int c, int& lo) {
  while (P.chunk_begin[lo + 1] <= c) ++lo;
  while (P.chunk_begin[lo] > c) --lo;
  Chunk C;
  C.i = lo;
  C.esize = P.numel[lo] < 0 ? 4 : 2;
  C.n = P.numel[lo] < 0 ? -P.numel[lo] : P.numel[lo];
  const uint8_t* base = static_cast<const uint8_t*>(P.grad[lo]);
  const int64_t head = (int64_t)(reinterpret_cast<uintptr_t>(base) & (kLine - 1));
  const int64_t off = (int64_t)(c - P.chunk_begin[lo]) * kChunkBytes - head;   // bytes from element 0
  C.e0 = off / C.esize;                 // exact: the head is a whole number of elements
  C.g = base + off;
  return C;
}

__device__ __forceinline__ uint4 load_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// The vector's 16 bytes, zero outside the tensor (values never read there).  CONST: the kernel does not
// write the tensor (clipping in place does, and the read-only path is for memory that nothing writes).
template <bool CONST>
__device__ __forceinline__ uint4 load_vec(const Chunk& C, int v) {
  const int per = 16 / C.esize;
  const int64_t e = C.e0 + (int64_t)v * per;
  const uint8_t* p = C.g + (int64_t)v * 16;
  if (e >= 0 && e + per <= C.n) return CONST ? ldg_nc_v4(p) : load_v4(p);
  uint32_t w[4] = {0, 0, 0, 0};
  if (e + per > 0 && e < C.n) {
    if (C.esize == 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e + k >= 0 && e + k < C.n) w[k] = reinterpret_cast<const uint32_t*>(p)[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (e + k >= 0 && e + k < C.n) w[k >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[k] << (16 * (k & 1));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ double sum_squares(const float (&x)[8]) {
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s = fmaf(x[k], x[k], s);
  // below 2^-60 a lost square (under 2^-149) could show in 53 bits' worth of the sum, zero
  // included; at FLT_MAX and above (or NaN) FP32 was too narrow
  if (s > 8.7e-19f && s < FLT_MAX) return (double)s;
  double d = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) d = fma((double)x[k], (double)x[k], d);
  return d;
}

__device__ __forceinline__ void unpack_bf16(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
  }
}

// Sum over the CTA, the same in every thread (fixed order: lanes, then warps).
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v += sh[w];
  return v;
}

__device__ __forceinline__ uint32_t bf16_rn(float x) {   // round to nearest even; NaN stays NaN
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

}  // namespace

template <int MAX>
__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const __grid_constant__ ClipTensors<MAX> P,
                                                             double* partials) {
  __shared__ double sh[kThreads / 32];
  double acc = 0.0;
  const int end = P.chunk_begin[P.n];
  int c = blockIdx.x, i = c < end ? tensor_of(P, c) : 0, esize = 4;
  uint4 next[kVecs];
  auto fetch = [&](int at) {
    const Chunk C = chunk_of(P, at, i);
    esize = C.esize;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) next[k] = load_vec<true>(C, k * kThreads + threadIdx.x);
  };
  if (c < end) fetch(c);
  for (; c < end; c += gridDim.x) {
    uint4 v[kVecs];
    const int es = esize;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) v[k] = next[k];
    if (c + (int)gridDim.x < end) fetch(c + gridDim.x);   // in flight under this chunk's squares
    if (es == 4) {
#pragma unroll
      for (int k = 0; k < kVecs; k += 2) {
        const float x[8] = {__uint_as_float(v[k].x), __uint_as_float(v[k].y), __uint_as_float(v[k].z),
                            __uint_as_float(v[k].w), __uint_as_float(v[k + 1].x), __uint_as_float(v[k + 1].y),
                            __uint_as_float(v[k + 1].z), __uint_as_float(v[k + 1].w)};
        acc += sum_squares(x);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        float x[8];
        unpack_bf16(v[k], x);
        acc += sum_squares(x);
      }
    }
  }
  acc = block_sum(acc, sh);
  if (threadIdx.x == 0) partials[blockIdx.x] = acc;
}

namespace {

// Writes the CTA's chunks, from the list's end, each value times coef: in FP32, or (SMALL: below
// FP32's normal range, where the factor itself would lose its bits) in FP64, rounded to FP32 once.
// Two loops, since a choice inside cost the FP32 one 4% (BF16 alone: 24%).
template <int MAX, bool SMALL>
__device__ __forceinline__ void scale_chunks(const ClipTensors<MAX>& P, double coef64) {
  const float coef = (float)coef64;
  auto times = [&](float x) { return SMALL ? (float)((double)x * coef64) : x * coef; };
  int c = P.chunk_begin[P.n] - 1 - (int)blockIdx.x;
  if (c < 0) return;
  int i = tensor_of(P, c);
  uint4 next[kVecs];
  Chunk N;
  auto fetch = [&](int at) {
    N = chunk_of(P, at, i);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) next[k] = load_vec<false>(N, k * kThreads + threadIdx.x);
  };
  fetch(c);
  for (; c >= 0; c -= gridDim.x) {
    const Chunk C = N;
    const int per = 16 / C.esize;
    uint4 v[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) v[k] = next[k];
    if (c >= (int)gridDim.x) fetch(c - gridDim.x);
    uint8_t* out = static_cast<uint8_t*>(P.out[C.i]) + C.e0 * C.esize;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      if (C.esize == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(times(__uint_as_float(w[j])));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bf16_rn(times(bf16_lo(w[j]))) | (bf16_rn(times(bf16_hi(w[j]))) << 16);
      }
      const int vec = k * kThreads + threadIdx.x;
      const int64_t e = C.e0 + (int64_t)vec * per;
      uint8_t* q = out + (int64_t)vec * 16;
      if (aligned && e >= 0 && e + per <= C.n) {
        __stcs(reinterpret_cast<uint4*>(q), make_uint4(w[0], w[1], w[2], w[3]));
      } else if (e + per > 0 && e < C.n) {
        if (C.esize == 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (e + j >= 0 && e + j < C.n) reinterpret_cast<uint32_t*>(q)[j] = w[j];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e + j >= 0 && e + j < C.n) reinterpret_cast<uint16_t*>(q)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
      }
    }
  }
}

}  // namespace

template <int MAX>
__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const __grid_constant__ ClipTensors<MAX> P,
                                                              const double* partials, int n_partials,
                                                              double max_norm, double eps, float* norm_out,
                                                              bool in_place) {
  __shared__ double sh[kThreads / 32];
  double t = 0.0;
  for (int k = threadIdx.x; k < n_partials; k += kThreads) t += partials[k];
  const double norm = sqrt(block_sum(t, sh));
  const double ratio = max_norm / (norm + eps);
  // no limit: the norm only; else a NaN norm gives a NaN factor
  const double coef = isinf(max_norm) || ratio >= 1.0 ? 1.0 : ratio;
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  if (in_place && (float)coef == 1.0f) return;             // 1 * g is g: nothing to write
  // gradients of 1e38 and a limit of 1, say
  if (coef > 0.0 && coef < (double)FLT_MIN) scale_chunks<MAX, true>(P, coef);
  else scale_chunks<MAX, false>(P, coef);
}

int clip_chunks(const void* grad, int64_t bytes) {
  return bytes == 0 ? 0 : (int)(((int64_t)(reinterpret_cast<uintptr_t>(grad) & (kLine - 1)) + bytes + kChunkBytes - 1) / kChunkBytes);
}

template <int MAX>
cudaError_t launch_clip_norm(const ClipTensors<MAX>& p, double* partials, int grid, cudaStream_t s) {
  clip_norm_kernel<MAX><<<grid, kThreads, 0, s>>>(p, partials);
  return cudaGetLastError();
}

template <int MAX>
cudaError_t launch_clip_scale(const ClipTensors<MAX>& p, const double* partials, int n_partials, double max_norm,
                              double eps, float* norm_out, bool in_place, int grid, cudaStream_t s) {
  clip_scale_kernel<MAX><<<grid, kThreads, 0, s>>>(p, partials, n_partials, max_norm, eps, norm_out, in_place);
  return cudaGetLastError();
}

template cudaError_t launch_clip_norm<kClipFew>(const ClipTensors<kClipFew>&, double*, int, cudaStream_t);
template cudaError_t launch_clip_norm<kClipMany>(const ClipTensors<kClipMany>&, double*, int, cudaStream_t);
template cudaError_t launch_clip_scale<kClipFew>(const ClipTensors<kClipFew>&, const double*, int, double, double,
                                                 float*, bool, int, cudaStream_t);
template cudaError_t launch_clip_scale<kClipMany>(const ClipTensors<kClipMany>&, const double*, int, double, double,
                                                  float*, bool, int, cudaStream_t);

}  // namespace fp8q
