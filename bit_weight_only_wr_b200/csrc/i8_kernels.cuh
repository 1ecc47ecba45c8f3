// Launch interface of the 8-bit token path: row quantizer, residual + norm, int8 product (internal to libwr).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "wr.h"

namespace wr {

// The status of a runtime call, reported here and not again by the next call that asks for the last error.
inline cudaError_t own_error(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// Launches a product so that it may start while the kernel before it in the stream still runs: its CTAs set up
// barriers and tensor memory and then wait in grid_dependency_wait() before they touch memory that
// another kernel may write or read. In a graph of such calls o of one token takes 2.9 us instead of
// 3.7, q/k/v of 32 tokens 6.2 instead of 7.5, down of 333 tokens 13.8 instead of 14.7; norm and q/k/v of
// 32 tokens together 9.0 instead of 10.6. (The row operators are launched plainly: their many small
// CTAs, started early, took slots from the kernel before; 8192 rows 45 instead of 40 us.)
template <typename... Params, typename... Args>
inline cudaError_t launch_overlapped(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream,
                                     const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return own_error(cudaLaunchKernelEx(&cfg, kern, args...));
}
// A launch in stream order. Its own status is returned, whatever calls before it left behind.
template <typename... Params, typename... Args>
inline cudaError_t launch_plain(void (*kern)(Params...), dim3 grid, dim3 block, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  return own_error(cudaLaunchKernelEx(&cfg, kern, args...));
}

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
constexpr int64_t kMaxNormDim = 32768;   // a row stays in one CTA

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
  int cut;         // persistent: pieces of each tile that is left over after whole rounds
  int tiles;
};
bool plan_gemm_i8(int64_t M, int64_t N, int64_t K, GemmI8Plan* p);   // false: too many tiles
// The kernel of a call. dp4a begins a second turn of rows behind 5328 of them (four in each of nine CTAs an SM),
// the warps' MMA behind 7104 (sixteen in each of three). dp4a's time goes by rows where they are short (0.31 us for a
// thousand of up to 1536 bytes), and by bytes where they are long. Measured in a graph of such calls, us (dp4a, warps'
// MMA, tcgen05):
//   one token   2560 x 4096: 2.9, 4.0, 5.9;  6144 x 1024: 3.5, 2.5, 3.9;  6144 x 2560: 4.3, 3.9, -;  6144 x 4096: 5.4, 6.0, -
//               8200 x 1024: 4.2, 4.0, 4.6;  16384 x 512: 6.6, 5.0, 4.3;  150000 x 1024: 47, 36, 27;  2560 x 1536: 2.4, 2.8, 4.1
//               9728 x 1536: 5.0, 4.7, 5.4;  40000 x 1040: 13.7, 14.1, 10.6;  40000 x 1536: 13.8, 12.4, 13.2
//               150000 x 1536: 48, 38, 37;   9728 x 2560: 5.8, 7.5, 6.9;  150000 x 2560: 57, 70, 59;  19456 x 9728: 32, 38, 31
//   2 tokens    2560 x 4096: 3.5, 3.9, 6.0;  6144 x 2560: 4.7, 3.9, -;    6144 x 9728: 13.0, 11.5, -;  5328 x 1536: 3.4, 3.1, 5.0
//               9728 x 1536: 5.7, 4.7, 5.4;  19456 x 2560: 10.8, 11.9, 10.3;  150000 x 2560: 66, 70, 60
//   8 tokens    2560 x 4096: -, 4.0, 5.2;    6144 x 9728: -, 11.5, 13.3;  8192 x 4096: -, 8.3, 8.7;  8192 x 5200: -, 12.4, 11.1
//               9728 x 512: -, 3.7, 3.3;     9728 x 1024: -, 4.2, 4.7;    19456 x 1024: -, 6.5, 6.1;  9728 x 2048: -, 5.7, 6.4
//               40000 x 2048: -, 14.7, 16.8; 150000 x 2048: -, 51, 51;    9728 x 2560: -, 7.4, 7.0;  150000 x 2560: -, 73, 62
//               19456 x 1536: -, 7.8, 7.5;   150000 x 1536: -, 42, 39
//   16 tokens   4096 x 4096: -, 5.0, 6.6;    6144 x 2560: -, 6.9, 6.0;    4736 x 6144: -, 7.2, 8.3;  2560 x 9728: -, 8.9, 8.2
//               4752 x 2048: -, 4.8, 5.4
// (9 to 16 tokens have two CTAs an SM: 4736 rows at once.) On 476 shapes of 1 to 16 tokens and up to 150000 rows the choice
// takes 1.0 % longer than the best of the three in the geometric mean.
enum class I8Kernel { kDp4a, kFew, kTcgen05 };
constexpr int kFewAtOnce = 148 * 3 * 16;
inline I8Kernel gemm_i8_kernel_for(int64_t M, int64_t N, int64_t K) {
  if (M <= 2 && (K > 2048 || N <= (K > 1024 ? 5328 : 1024))) {
    const bool second_turn = N > 5328 && N <= kFewAtOnce;
    return second_turn && (M == 2 || K <= 2560) ? I8Kernel::kFew : I8Kernel::kDp4a;
  }
  if (M <= 8 && (N <= kFewAtOnce || (N <= 8192 && K <= 4096) || (K <= 2048 && K >= (N <= 12288 ? 1024 : 1792)))) return I8Kernel::kFew;
  if (M <= 16 && N <= kFewAtOnce / 3 * 2 && K <= 6144) return I8Kernel::kFew;
  return I8Kernel::kTcgen05;
}
cudaError_t launch_gemv_i8(const GemmI8Args& a, cudaStream_t stream);   // M <= 2
cudaError_t launch_few_i8(const GemmI8Args& a, cudaStream_t stream);    // M <= 16
constexpr uint64_t kGemmWaitNs = 1000000000ull;   // limit of a wait in the tcgen05 forms
cudaError_t launch_gemm_i8(const GemmI8Args& a, const GemmI8Plan& p, int* err, cudaStream_t stream, uint64_t wait_ns = kGemmWaitNs);
// Sums of K products of int8 values stay inside int32 up to this K ((-128)^2 * K < 2^31).
constexpr int64_t kMaxI8K = 131071;

}  // namespace wr
