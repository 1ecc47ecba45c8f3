// Launch interface of the 8-bit token path: row quantizer, residual + norm, int8 product (internal to libwr).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "wr.h"

namespace wr {

// Row quantizer: v = x (or silu(gate) x), one fp32 scale and int8 codes per row.
struct QuantRowsArgs {
  const uint8_t* x;
  const uint8_t* gate;       // null: v = x
  int8_t* q;
  float* scale;
  int64_t ldx, ldg, ldq;     // in elements
  int64_t M;
  int K;
  int type;                  // WR_F32 / WR_BF16 / WR_F16, of x and gate
};
cudaError_t launch_quantize_rows(const QuantRowsArgs& a, cudaStream_t stream);

// Residual + norm around a block (wr_residual_norm_args, checked).
cudaError_t launch_residual_norm(const wr_residual_norm_args& a, cudaStream_t stream);
constexpr int64_t kMaxNormDim = 32768;   // a row's values stay in the registers of one CTA

// Int8 product.
struct GemmI8Args {
  const int8_t* x;           // [M, ldx]
  const int8_t* w;           // [N, ldw]
  const float* x_scale;      // [M]
  const float* w_scale;      // [N]
  const float* bias;         // [N] or null
  void* y;                   // [M, ldy] of y_type
  int64_t ldx, ldw, ldy;
  int M, N, K;
  int y_type;
};
// The work of one call on the tensor cores, planned on the host (see gemm_i8.cu).
struct GemmI8Plan {
  int pair;        // 1: CTA pairs (256 channels a tile), 0: single CTAs (128)
  int persistent;  // 1: pairs that take tiles in turn, 0: a cluster for each tile
  int tn;          // tokens a tile
  int mt;          // token tiles
  int kb;          // 128-byte blocks of K
  int split;       // parts of a tile's K
  int tiles;
};
bool plan_gemm_i8(int64_t M, int64_t N, int64_t K, GemmI8Plan* p);   // false: too many tiles
// Tokens up to which the product runs on dp4a, without a workspace.
constexpr int kGemvI8Tokens = 2;
cudaError_t launch_gemv_i8(const GemmI8Args& a, cudaStream_t stream);
cudaError_t launch_gemm_i8(const GemmI8Args& a, const GemmI8Plan& p, int* err, cudaStream_t stream);
// Sums of K products of int8 values stay inside int32 up to this K ((-128)^2 * K < 2^31).
constexpr int64_t kMaxI8K = 131071;

}  // namespace wr
