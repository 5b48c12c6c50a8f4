// Host-side launch interfaces of the kernels (internal to the library).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fp8q {

enum { kTile1x128 = 0, kTile128 = 1, kTileMX = 2 };

struct TileQuantParams {
  const uint16_t* x;
  int64_t rows, cols, ld_x;
  uint8_t* q_row;
  void* s_row;      // float* (1x128, 128x128) or uint8_t* (MX)
  int64_t ld_s_row;  // 1x128: scale row stride; 128x128: K/128
  uint8_t* q_col;
  void* s_col;
  int64_t ld_s_col;
  int tiles_c;      // 128-column tiles per 128-row band
  int sf_tiled;     // MX scale bytes in the MMA-tiled layout
  // grouped calls (0 = one matrix): tiles per matrix, and each operand's stride between
  // consecutive matrices (x in elements, outputs and scales in bytes)
  int64_t batch_tiles;
  int64_t x_bstride, q_row_bstride, q_col_bstride, s_row_bstride, s_col_bstride;
};

cudaError_t launch_tile_quant(int mode, bool row, bool col, const TileQuantParams& p,
                              int64_t tiles, cudaStream_t s);

// Multi-tensor launch: up to kMaxMultiItems tensors, each a 1x128 (rowwise, colwise or both)
// or a 128x128 (either or both layouts) quantization; item i owns the launch's tiles
// [tile_begin[i], tile_begin[i + 1]).
constexpr int kMaxMultiItems = 8;
enum { kMulti1x128Row = 0, kMulti1x128Col = 1, kMulti1x128Both = 2, kMulti128Row = 3, kMulti128Col = 4,
       kMulti128Both = 5 };
struct TileQuantMulti {
  int n;
  int kind[kMaxMultiItems];
  int64_t tile_begin[kMaxMultiItems + 1];
  TileQuantParams item[kMaxMultiItems];
};
cudaError_t launch_tile_quant_multi(const TileQuantMulti& m, int64_t tiles, cudaStream_t s);

// 1x128 quantization grouped by expert (`groups` of them, row offsets on the device): the
// transposed output has `bands` bands of 128 columns; codes of rows, if `row`, as ungrouped.
cudaError_t launch_tile_quant_grouped(bool row, const TileQuantParams& p, const int32_t* offs, int groups,
                                      int64_t bands, int num_sms, uint32_t* status, cudaStream_t s);

// Per-tensor current scaling: amax pass into *amax_bits (zeroed by the caller), then cast.
cudaError_t launch_tensor_amax(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                               uint32_t* amax_bits, cudaStream_t s);
cudaError_t launch_tensor_cast(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                               const uint32_t* amax_bits, uint8_t* q, float* s_dec,
                               cudaStream_t s);

struct Fp4QuantParams {
  const uint16_t* x;
  int64_t rows, cols, ld_x;
  int rht_row, rht_col, sr_row, sr_col;
  uint32_t rht_k0, rht_k1, sr_k0, sr_k1;
  uint8_t* q_row;
  uint8_t* sf_row;
  float* g_row;
  uint8_t* q_col;
  uint8_t* sf_col;
  float* g_col;
  int sf_tiled;
  int tiles_c;
  uint32_t* amax_bits;  // [0]: rowwise output's global amax, [1]: colwise output's
  uint32_t sr_rk[20];   // Philox key schedule of the stochastic-rounding key (sr_k0, sr_k1)
};

// One float written on the stream (the decode scale of an empty tensor), no host sync.
cudaError_t launch_fill_f32(float* dst, float v, cudaStream_t s);

cudaError_t launch_tensor_delayed(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, float* hist,
                                  int hlen, int pos, bool e5m2, uint8_t* q, float* s_dec, uint32_t* amax_bits,
                                  cudaStream_t s);

cudaError_t launch_fp4_amax(const Fp4QuantParams& p, int64_t tiles, cudaStream_t s);
cudaError_t launch_fp4_quant(const Fp4QuantParams& p, int64_t tiles, cudaStream_t s);
// 16x16-block weight quantizer: global amax into amax_bits[0], then codes in the layouts
// whose q pointer is set; g_row receives the decode scale.
cudaError_t launch_fp4_quant_2d(const Fp4QuantParams& p, int64_t tiles, cudaStream_t s);

// ------------------------------------------------------------------ gradient norm and clipping
// Up to MAX tensors of one launch, passed by value (a launch of few tensors passes few bytes;
// kernel parameters hold 32764 bytes): numel is negative for FP32, positive for BF16; tensor i
// owns the launch's 16 KB chunks [chunk_begin[i], chunk_begin[i + 1]).
constexpr int kClipFew = 64, kClipMany = 1024;
template <int MAX>
struct ClipTensors {
  int n;
  int chunk_begin[MAX + 1];
  const void* grad[MAX];
  void* out[MAX];
  int64_t numel[MAX];
};
static_assert(sizeof(ClipTensors<kClipMany>) + 64 <= 32764, "kernel parameters");
// Chunks of a tensor (their first starts at the 128-byte line that its first element is in).
int clip_chunks(const void* grad, int64_t bytes);
// partials[0 .. grid): each CTA's sum of squares.
template <int MAX>
cudaError_t launch_clip_norm(const ClipTensors<MAX>& p, double* partials, int grid, cudaStream_t s);
// norm = sqrt(sum of all partials) into norm_out (unless NULL), then out = min(1, max_norm /
// (norm + eps)) * grad; in_place: every out is its grad.
template <int MAX>
cudaError_t launch_clip_scale(const ClipTensors<MAX>& p, const double* partials, int n_partials, double max_norm,
                              double eps, float* norm_out, bool in_place, int grid, cudaStream_t s);

// ------------------------------------------------------------------ norms around a block
// Forward: y, h -> h_out, n_out and / or q_row, s_row; backward: dn, dh_in, y, h (the stored
// h') -> dh, dy and the column sums.  Leading dimensions in elements.
struct NormParams {
  int64_t rows;
  int cols, stages;   // stages: rows staged in shared memory (set by the launcher)
  float alpha, eps;
  const void *y, *h, *w_post, *gate, *w_pre, *dn, *dh_in;
  int64_t ld_y, ld_h, ld_dn, ld_dh_in;
  void *h_out, *n_out, *dh, *dy;
  int64_t ld_h_out, ld_n, ld_dh, ld_dy;
  uint8_t* q_row;
  float* s_row;
  int64_t ld_s_row;
  float *rstd_post, *rstd_pre;
  float *dw_pre, *dw_post, *dgate;
  float* partials;    // [norm_backward_ctas][2][cols]
  uint32_t* status;
};
int norm_backward_ctas(int64_t rows, int cols, bool h32, int num_sms);
cudaError_t launch_norm_forward(const NormParams& p, bool h32, bool w32, int num_sms, cudaStream_t s);
cudaError_t launch_norm_backward(const NormParams& p, bool h32, bool w32, int num_sms, cudaStream_t s);

// ------------------------------------------------------------------ GEMM
// Output tile width of the blockwise (FP32-promotion) kernel; the B and wgrad-scale TMA boxes
// are built with it.
constexpr uint32_t kBlockwiseTileN = 256;

struct GemmParams {
  int recipe;       // fp8q_recipe
  int layout;       // fp8q_layout
  int M, N, K;
  const float* sa;  // BLOCKWISE: A decode scales, sa[kb * ld_sa + m]
  int64_t ld_sa;
  const float* sb;  // BLOCKWISE: B scales (indexed per layout)
  int64_t ld_sb;
  const float* a_global;
  const float* b_global;
  uint16_t* c;      // BF16 row-major (nullptr when accumulating into c32)
  float* c32;       // BLOCKWISE FP32 accumulate target (C += A.B^T), else nullptr
  int64_t ldc;
  const uint8_t* sfa;  // MX / NVFP4: MMA-tiled scale images
  const uint8_t* sfb;
  int64_t sfa_s4, sfb_s4;  // atoms per 128-row band (ceil(scale columns / 4))
  const int32_t* m_offsets;
  int num_groups;
  int tiles_m, tiles_n;    // output tile grid (non-grouped)
  int group_m;             // raster: row tiles per column sweep (set by the launcher)
  int group_n;             // raster: > 0 -> column tiles per row sweep instead (set by the launcher)
  int a_fmt, b_fmt;        // PERTENSOR: element format of A / B (0 E4M3, 1 E5M2)
  uint8_t* q_out;          // BLOCKWISE, optional: 1x128 E4M3 codes of the BF16 output (along N)
  float* s_out;            //   and their decode scales, s_out[(n / 128) * ld_s_out + m]
  int64_t ld_q_out, ld_s_out;
  uint32_t* status;        // device status word
  // BLOCKWISE, not grouped (set by the launcher): units [0, main_tiles) are the
  // whole raster tiles; with tail_splits > 0 the remaining tiles (the last, partial wave)
  // follow as tail_splits K ranges each, whose FP32 partial sums go to ws (256 x 256 floats
  // per range) and are then added by a second kernel.
  int main_tiles;
  int tail_splits;
  float* ws;
  int64_t ws_bytes;
};

cudaError_t launch_selftest_wait(uint32_t* status, uint64_t limit_ns, cudaStream_t s);

// tma_c: C for the blockwise kernel's epilogues, N inner, M outer: BF16 with 32 x 32 boxes
// (stored), or FP32 with 16 x 32 boxes (added, FP32 accumulation), 64-byte swizzle; for grouped
// GEMMs boxes twice as wide, 64 x 32 or 32 x 32, and 128-byte swizzle; tma_q: the fused
// quantization's E4M3 codes (64 x 32 boxes, stored); tma_ws: p.ws as FP32 rows of 256 (16 x 32
// boxes, 64-byte swizzle), used only when the last wave is split (in place of
// tma_q, which the BF16 and FP32-accumulate epilogues do not use).
cudaError_t launch_gemm(const GemmParams& p, const CUtensorMap& tma_a, const CUtensorMap& tma_b,
                        const CUtensorMap& tma_sb, const CUtensorMap& tma_c, const CUtensorMap& tma_q,
                        const CUtensorMap& tma_ws, int num_sms, cudaStream_t s);

// Grouped fprop / dgrad with few rows per expert: its own kernel (gemm_rows.cu), with TMA boxes
// of this many rows of A (0: the large kernel) and 128 rows of B.  Defined in gemm_rows.cu.
int gemm_few_rows_tile(int64_t M, int64_t N, int groups, int num_sms);
cudaError_t launch_gemm_few_rows(const GemmParams& p, const CUtensorMap& tma_a, const CUtensorMap& tma_w, int num_sms,
                                 cudaStream_t s);

// Workspace bytes that a blockwise BF16 GEMM with these parameters uses to split its last,
// partial wave into K ranges on the current device (0: it would not split).
size_t blockwise_workspace_bytes(const GemmParams& p, int num_sms);

}  // namespace fp8q
