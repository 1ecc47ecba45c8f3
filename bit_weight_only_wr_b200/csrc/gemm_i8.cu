// Int8 product with a scale for each token and each output channel (sm_100a):
//   y[m,n] = (sum_k x[m,k] w[n,k]) x_scale[m] w_scale[n] + bias[n]
// The sums are exact 32-bit integers (K <= 131071), so that they do not depend on the order or on how
// K is split; the conversion and the two products are fp32, in this order, in every kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "i8_kernels.cuh"

namespace wr {
namespace {

__device__ __forceinline__ float scaled(int acc, float xs, float ws, const float* bias, int n) {
  const float v = (float)acc * xs * ws;
  return bias ? v + __ldg(bias + n) : v;
}
__device__ __forceinline__ void store_y(void* y, int type, int64_t at, float v) {
  if (type == WR_F32) static_cast<float*>(y)[at] = v;
  else if (type == WR_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// ---------------------------------------------------------------- few tokens: dp4a, one pass over w

// The 16 bytes at k of a row of K bytes, zero behind its end (nothing behind the row is read).
template <bool STREAM>
__device__ __forceinline__ uint4 row_chunk(const int8_t* row, int k, int K) {
  if (k + 16 <= K) {
    if (STREAM) return ld_stream_v4(row + k);
    return __ldg(reinterpret_cast<const uint4*>(row + k));
  }
  uint32_t w[4] = {0, 0, 0, 0};
  for (int i = 0; i < 16; ++i) {
    if (k + i < K) {
      const uint32_t b = (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
      if (i < 4) w[0] |= b;
      else if (i < 8) w[1] |= b;
      else if (i < 12) w[2] |= b;
      else w[3] |= b;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int acc) {
  acc = __dp4a((int)a.x, (int)b.x, acc);
  acc = __dp4a((int)a.y, (int)b.y, acc);
  acc = __dp4a((int)a.z, (int)b.z, acc);
  return __dp4a((int)a.w, (int)b.w, acc);
}

// A warp owns R rows of w and MT tokens and reads the rows once, 512 bytes of each a step; x stays in
// L1. grid.y covers the tokens in steps of MT.
template <int R, int MT>
__global__ void __launch_bounds__(128) gemv_i8_kernel(const GemmI8Args a) {
  const int lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * R, m0 = blockIdx.y * MT;
  if (n0 >= a.N) return;
  const int8_t *w[R], *x[MT];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw;
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = a.x + (int64_t)min(m0 + m, a.M - 1) * a.ldx;
  int acc[R][MT] = {};
  constexpr int U = 8 / R;   // row loads in flight: 8 a lane
  for (int k0 = 0; k0 < a.K; k0 += 512 * U) {
    uint4 wv[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int k = k0 + 512 * u + 16 * lane;
        wv[u][r] = k < a.K ? row_chunk<true>(w[r], k, a.K) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 512 * u + 16 * lane;
      if (k >= a.K) break;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 xv = row_chunk<false>(x[m], k, a.K);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][m] = dot16(wv[u][r], xv, acc[r][m]);
      }
    }
  }
  // lane r + R m keeps the sum of row r and token m
  int mine = 0;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int s = __reduce_add_sync(0xffffffffu, acc[r][m]);
      if (lane == r + R * m) mine = s;
    }
  const int n = n0 + lane % R, m = m0 + lane / R;
  if (lane < R * MT && n < a.N && m < a.M)
    store_y(a.y, a.y_type, (int64_t)m * a.ldy + n, scaled(mine, __ldg(a.x_scale + m), __ldg(a.w_scale + n), a.bias, n));
}

template <int R, int MT>
cudaError_t run_gemv(const GemmI8Args& a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.N + 4 * R - 1) / (4 * R)), (unsigned)((a.M + MT - 1) / MT));
  gemv_i8_kernel<R, MT><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemv_i8(const GemmI8Args& a, cudaStream_t stream) {
  if (a.M == 1) return run_gemv<1, 1>(a, stream);
  if (a.M == 2) return run_gemv<2, 2>(a, stream);
  if (a.M <= 4) return run_gemv<4, 4>(a, stream);
  return run_gemv<4, 8>(a, stream);
}

}  // namespace wr
