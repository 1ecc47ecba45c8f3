// Row operators of the 8-bit token path (sm_100a): the row quantizer, and the residual + norm that
// joins one block's output to the next block's input.
//
//   quantize:  v = x, or silu(g) x;  A = max_k |v_k|;  s = A / 127;  q_k = nearest integer to 127 v_k / A
//   norm:      h' = r h + g * post(b),  post(b) = b or b / sqrt(mean b^2 + eps) * w_post
//              y  = h' / sqrt(mean h'^2 + eps) * w   (bf16, fp16, fp32, or quantized as above)
//
// Both are bound by memory: every input is read once and every output written once. One CTA owns a
// row and keeps its values in registers between the reductions, so that nothing is read twice; a
// thread holds VPT vectors of 8 elements. All arithmetic is fp32 and rounds once to the output's type.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "i8_kernels.cuh"

namespace wr {
namespace {

// ---------------------------------------------------------------- loads and stores of 8 elements

// Eight elements as loaded: 16 bytes of a 16-bit type (a), 32 bytes of fp32 (a, b). Loads are issued
// for all operands of a row before the first is converted, so they are kept raw.
struct Raw8 {
  uint32_t r[8];
};

__device__ __forceinline__ uint4 ld16(const uint8_t* p, bool pred) {
  uint4 v = make_uint4(0, 0, 0, 0);
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
               : "l"(p), "r"((int)pred));
  return v;
}

// Where element j of vector i of thread t sits in its row. VEC: 8 neighbours; otherwise (rows that
// do not start on 16 bytes) neighbouring threads take neighbouring elements, one load each.
template <bool VEC>
__device__ __forceinline__ int elem(int i, int j, int T, int t) {
  return VEC ? (i * T + t) * 8 + j : (i * 8 + j) * T + t;
}

template <bool VEC>
__device__ __forceinline__ Raw8 load8(const uint8_t* row, int type, int i, int T, int t, int D) {
  Raw8 v;
  const bool f32 = type == WR_F32;
  if (VEC) {
    const int e = elem<true>(i, 0, T, t);
    const bool whole = e + 8 <= D;
    const uint8_t* p = row + (int64_t)e * (f32 ? 4 : 2);
    const uint4 a = ld16(p, whole), b = ld16(p + 16, whole && f32);
    v.r[0] = a.x; v.r[1] = a.y; v.r[2] = a.z; v.r[3] = a.w;
    v.r[4] = b.x; v.r[5] = b.y; v.r[6] = b.z; v.r[7] = b.w;
    if (!whole && e < D) {   // the row's last vector
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (e + j < D) {
          if (f32) v.r[j] = reinterpret_cast<const uint32_t*>(row)[e + j];
          else v.r[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[e + j] << (16 * (j & 1));
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v.r[j] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = elem<false>(i, j, T, t);
      if (e < D) {
        if (f32) v.r[j] = reinterpret_cast<const uint32_t*>(row)[e];
        else v.r[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[e] << (16 * (j & 1));
      }
    }
  }
  return v;
}

__device__ __forceinline__ void to_float8(const Raw8& v, int type, float f[8]) {
  if (type == WR_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v.r[j]);
  } else if (type == WR_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(v.r[j] << 16);
      f[2 * j + 1] = __uint_as_float(v.r[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&v.r[j]));
      f[2 * j] = h.x;
      f[2 * j + 1] = h.y;
    }
  }
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int type) {
  if (type == WR_BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rounds to nearest even (fp16 beyond 65504 gives infinity, as the type does).
template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* row, int type, int i, int T, int t, int D, const float f[8]) {
  uint32_t p[4];
  if (type != WR_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = pack16(f[2 * j], f[2 * j + 1], type);
  }
  const int e0 = elem<VEC>(i, 0, T, t);
  if (VEC && e0 + 8 <= D) {
    if (type == WR_F32) {
      float4* o = reinterpret_cast<float4*>(row + (int64_t)e0 * 4);
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(row + (int64_t)e0 * 2) = make_uint4(p[0], p[1], p[2], p[3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = elem<VEC>(i, j, T, t);
    if (e < D) {
      if (type == WR_F32) reinterpret_cast<float*>(row)[e] = f[j];
      else reinterpret_cast<uint16_t*>(row)[e] = (uint16_t)(p[j / 2] >> (16 * (j & 1)));
    }
  }
}

// ---------------------------------------------------------------- reductions over a row's CTA

// Every warp leaves its value in buf and every thread reads all of them: one barrier for each
// reduction (each has its own buf). The sum runs in the same order in every thread and every run.
__device__ __forceinline__ float row_sum(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = (threadIdx.x & 31) < nw ? buf[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// Largest magnitude, by its bits: an infinity is above every number and a NaN above that.
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* buf) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < nw ? buf[threadIdx.x & 31] : 0u);
}

// ---------------------------------------------------------------- the 8-bit rounding

// Codes of one row with largest magnitude A: the integer nearest to 127 v / A, a tie to the even one,
// decided on the exact quotient. t = v * fl(127 / A) is off by at most 127 * 2^-23 < 1.6e-5 (two
// roundings of at most 2^-24 relative each), so only a value that close to the middle of two codes
// needs more: there the quotient is formed in fp64. The 31-bit product 127 v is exact in fp64, a tie's
// quotient is exact too, and any other quotient is at least 2^-40 (relative) away from a tie.
// A = 0: codes 0 and scale 0. A not finite (an infinity or NaN in the row): codes 0 and scale NaN, so
// that whatever is computed from the row is NaN. Below 2^-100 fl(127 / A) could overflow: all in fp64.
struct RowCode {
  float A, inv, scale;
  bool wide;
};
__device__ __forceinline__ RowCode row_code(uint32_t amax_bits) {
  RowCode c;
  c.A = __uint_as_float(amax_bits);
  const bool finite = amax_bits < 0x7F800000u;
  c.wide = finite && c.A > 0.f && c.A < 7.8886090522e-31f;
  c.inv = finite && c.A > 0.f && !c.wide ? __fdiv_rn(127.f, c.A) : 0.f;
  c.scale = finite ? __fdiv_rn(c.A, 127.f) : __uint_as_float(0x7FC00000u);
  if (!finite) c.A = 0.f;
  return c;
}
__device__ __noinline__ float code_exact(float v, float A) { return (float)rint((double)v * 127.0 / (double)A); }
__device__ __forceinline__ int code_of(const RowCode& c, float v) {
  if (c.A == 0.f) return 0;
  const float t = v * c.inv;
  float r = rintf(t);
  if (c.wide || fabsf(fabsf(t - r) - 0.5f) < 2e-5f) r = code_exact(v, c.A);
  return (int)r;
}

template <bool VEC>
__device__ __forceinline__ void store_codes8(int8_t* row, int i, int T, int t, int D, const RowCode& c, const float f[8]) {
  uint32_t p[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) p[j / 4] |= (uint32_t)(code_of(c, f[j]) & 0xFF) << (8 * (j & 3));
  const int e0 = elem<VEC>(i, 0, T, t);
  if (VEC && e0 + 8 <= D) {
    *reinterpret_cast<uint2*>(row + e0) = make_uint2(p[0], p[1]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = elem<VEC>(i, j, T, t);
    if (e < D) row[e] = (int8_t)(p[j / 4] >> (8 * (j & 3)));
  }
}

__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + expf(-g)); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ---------------------------------------------------------------- row quantizer

// VPT > 0: the row stays in registers. VPT = 0: rows longer than that; read twice (the second time
// mostly from L2), VEC in steps of one vector.
template <int VPT, int MAXT, bool VEC>
__global__ void __launch_bounds__(MAXT) quantize_rows_kernel(const QuantRowsArgs a) {
  __shared__ uint32_t buf[32];
  const int T = blockDim.x, t = threadIdx.x;
  const int64_t m = blockIdx.x;
  const int es = a.type == WR_F32 ? 4 : 2;
  const uint8_t* x = a.x + m * a.ldx * es;
  const uint8_t* g = a.gate ? a.gate + m * a.ldg * es : nullptr;
  int8_t* q = a.q + m * a.ldq;
  auto values = [&](const Raw8& rx, const Raw8& rg, float f[8]) {
    to_float8(rx, a.type, f);
    if (g) {
      float gf[8];
      to_float8(rg, a.type, gf);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= silu(gf[j]);
    }
  };
  uint32_t amax = 0;
  if constexpr (VPT > 0) {
    Raw8 rx[VPT], rg[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      rx[i] = load8<VEC>(x, a.type, i, T, t, a.K);
      if (g) rg[i] = load8<VEC>(g, a.type, i, T, t, a.K);
    }
    float f[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      values(rx[i], rg[i], f[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(f[i][j]));
    }
    const RowCode c = row_code(row_max(amax, buf));
#pragma unroll
    for (int i = 0; i < VPT; ++i) store_codes8<VEC>(q, i, T, t, a.K, c, f[i]);
    if (t == 0) a.scale[m] = c.scale;
  } else {
    const int steps = (a.K + 8 * T - 1) / (8 * T);
    float f[8];
    for (int i = 0; i < steps; ++i) {
      const Raw8 rx = load8<VEC>(x, a.type, i, T, t, a.K);
      Raw8 rg = rx;
      if (g) rg = load8<VEC>(g, a.type, i, T, t, a.K);
      values(rx, rg, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(f[j]));
    }
    const RowCode c = row_code(row_max(amax, buf));
    for (int i = 0; i < steps; ++i) {
      const Raw8 rx = load8<VEC>(x, a.type, i, T, t, a.K);
      Raw8 rg = rx;
      if (g) rg = load8<VEC>(g, a.type, i, T, t, a.K);
      values(rx, rg, f);
      store_codes8<VEC>(q, i, T, t, a.K, c, f);
    }
    if (t == 0) a.scale[m] = c.scale;
  }
}

// ---------------------------------------------------------------- residual + norm

__host__ __device__ inline int type_bytes(int type) { return type == WR_F32 ? 4 : (type == WR_I8 ? 1 : 2); }

template <int VPT, int MAXT, bool VEC>
__global__ void __launch_bounds__(MAXT) residual_norm_kernel(const wr_residual_norm_args a) {
  __shared__ float buf_post[32], buf_norm[32];
  __shared__ uint32_t buf_max[32];
  const int T = blockDim.x, t = threadIdx.x, D = (int)a.D;
  const int64_t m = blockIdx.x;
  auto row_of = [&](const void* p, int64_t ld, int type) {
    return static_cast<const uint8_t*>(p) + m * ld * type_bytes(type);
  };
  const uint8_t* b = a.block ? row_of(a.block, a.ld_block, a.block_type) : nullptr;
  const uint8_t* h = a.residual ? row_of(a.residual, a.ld_residual, a.residual_type) : nullptr;
  const uint8_t* g = a.gate ? row_of(a.gate, a.ld_gate, a.gate_type) : nullptr;
  const float inv_d = 1.f / (float)D;
  float v[VPT][8];   // the block's output, then h'
  // the row itself is loaded at once; the gate and the weights too where the registers allow it
  // (otherwise when they are used: they are the same for all rows and come from L2)
  constexpr bool kEarly = VPT == 1;
  Raw8 rb[VPT], rh[VPT], rg[VPT], rp[VPT], rn[VPT];
  const uint8_t* pw = static_cast<const uint8_t*>(a.post_norm ? a.post_weight : nullptr);
  const uint8_t* nw = static_cast<const uint8_t*>(a.y ? a.norm_weight : nullptr);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (b) rb[i] = load8<VEC>(b, a.block_type, i, T, t, D);
    if (h) rh[i] = load8<VEC>(h, a.residual_type, i, T, t, D);
    if (kEarly && pw) rp[i] = load8<VEC>(pw, a.weight_type, i, T, t, D);
    if (kEarly && g) rg[i] = load8<VEC>(g, a.gate_type, i, T, t, D);
    if (kEarly && nw) rn[i] = load8<VEC>(nw, a.weight_type, i, T, t, D);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (b) to_float8(rb[i], a.block_type, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
  }
  if (a.post_norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    const float r = 1.f / sqrtf(row_sum(ss, buf_post) * inv_d + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[8];
      if (pw) {
        if (!kEarly) rp[i] = load8<VEC>(pw, a.weight_type, i, T, t, D);
        to_float8(rp[i], a.weight_type, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * (w[j] + a.weight_offset);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= r;
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (g) {
      float w[8];
      if (!kEarly) rg[i] = load8<VEC>(g, a.gate_type, i, T, t, D);
      to_float8(rg[i], a.gate_type, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= w[j];
    }
    if (h) {
      float w[8];
      to_float8(rh[i], a.residual_type, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(a.residual_scale, w[j], v[i][j]);
    }
    if (a.residual_out)
      store8<VEC>(static_cast<uint8_t*>(a.residual_out) + m * a.ld_residual_out * type_bytes(a.residual_type),
                  a.residual_type, i, T, t, D, v[i]);
    // elements past the row are zero times whatever was loaded there (zero): they add nothing
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  if (!a.y) return;
  const float r = 1.f / sqrtf(row_sum(ss, buf_norm) * inv_d + a.eps);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (nw) {
      float w[8];
      if (!kEarly) rn[i] = load8<VEC>(nw, a.weight_type, i, T, t, D);
      to_float8(rn[i], a.weight_type, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * (w[j] + a.weight_offset);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= r;
    }
    if (a.y_type == WR_I8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (elem<VEC>(i, j, T, t) < D) amax = max(amax, abs_bits(v[i][j]));
    } else {
      store8<VEC>(static_cast<uint8_t*>(a.y) + m * a.ld_y * type_bytes(a.y_type), a.y_type, i, T, t, D, v[i]);
    }
  }
  if (a.y_type == WR_I8) {
    const RowCode c = row_code(row_max(amax, buf_max));
    int8_t* q = static_cast<int8_t*>(a.y) + m * a.ld_y;
#pragma unroll
    for (int i = 0; i < VPT; ++i) store_codes8<VEC>(q, i, T, t, D, c, v[i]);
    if (t == 0) a.y_scale[m] = c.scale;
  }
}

inline bool rows_aligned(int64_t M, int64_t ld, int bytes) { return M == 1 || ld * bytes % 16 == 0; }

// Threads that hold a row of D elements, VPT vectors of 8 each.
inline int row_threads(int64_t D, int vpt) { return (int)std::min<int64_t>(1024, ((D + 8 * vpt - 1) / (8 * vpt) + 31) / 32 * 32); }

}  // namespace

cudaError_t launch_quantize_rows(const QuantRowsArgs& a, cudaStream_t stream) {
  const int es = type_bytes(a.type);
  const bool vec = rows_aligned(a.M, a.ldx, es) && (!a.gate || rows_aligned(a.M, a.ldg, es)) && (a.M == 1 || a.ldq % 8 == 0);
  const unsigned grid = (unsigned)a.M;
#define WR_QUANT(VPT, MAXT)                                                                                  \
  do {                                                                                                       \
    const int T = row_threads(a.K, VPT > 0 ? VPT : 4);                                                       \
    if (vec) quantize_rows_kernel<VPT, MAXT, true><<<grid, T, 0, stream>>>(a);                               \
    else quantize_rows_kernel<VPT, MAXT, false><<<grid, T, 0, stream>>>(a);                                  \
  } while (0)
  if (a.K <= 4096) WR_QUANT(1, 512);
  else if (a.K <= 8192) WR_QUANT(2, 512);
  else if (a.K <= 16384) WR_QUANT(4, 512);
  else if (a.K <= 32768) WR_QUANT(4, 1024);
  else WR_QUANT(0, 1024);
#undef WR_QUANT
  return cudaGetLastError();
}

cudaError_t launch_residual_norm(const wr_residual_norm_args& a, cudaStream_t stream) {
  const bool vec = (!a.block || rows_aligned(a.M, a.ld_block, type_bytes(a.block_type))) &&
                   (!a.residual || rows_aligned(a.M, a.ld_residual, type_bytes(a.residual_type))) &&
                   (!a.residual_out || rows_aligned(a.M, a.ld_residual_out, type_bytes(a.residual_type))) &&
                   (!a.gate || rows_aligned(a.M, a.ld_gate, type_bytes(a.gate_type))) &&
                   (!a.y || (a.y_type == WR_I8 ? a.M == 1 || a.ld_y % 8 == 0 : rows_aligned(a.M, a.ld_y, type_bytes(a.y_type))));
  const unsigned grid = (unsigned)a.M;
#define WR_NORM(VPT, MAXT)                                                                                   \
  do {                                                                                                       \
    const int T = row_threads(a.D, VPT);                                                                     \
    if (vec) residual_norm_kernel<VPT, MAXT, true><<<grid, T, 0, stream>>>(a);                               \
    else residual_norm_kernel<VPT, MAXT, false><<<grid, T, 0, stream>>>(a);                                  \
  } while (0)
  if (a.D <= 4096) WR_NORM(1, 512);
  else if (a.D <= 8192) WR_NORM(2, 512);
  else if (a.D <= 16384) WR_NORM(4, 512);
  else WR_NORM(4, 1024);
#undef WR_NORM
  return cudaGetLastError();
}

}  // namespace wr
