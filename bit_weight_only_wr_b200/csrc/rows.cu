// Row operators of the 8-bit token path (sm_100a): the row quantizer, and the residual + norm that
// joins one block's output to the next block's input.
//
//   quantize:  v = x, or silu(g) x;  A = max_k |v_k|;  s = A / 127;  q_k = nearest integer to 127 v_k / A
//   norm:      h' = r h + g * post(b),  post(b) = b or b / sqrt(mean b^2 + eps) * w_post
//              y  = h' / sqrt(mean h'^2 + eps) * w   (bf16, fp16, fp32, or quantized as above)
//
// Both are bound by memory: every input is read once and every output written once. One CTA owns a
// row and keeps its values in registers between the reductions, so that nothing is read twice; a
// thread holds VPT vectors of 8 elements. Not all of a norm's fit where a row is longer than 16384: four
// vectors of each operand in 64 registers (1024 threads) leave 0.25 to 1.4 KB a thread in local memory, and
// 1000 bf16 rows of 20000 take 82 us and of 32768 121, of 16384 43. Quantizer rows of more than 32768 are read
// twice: 1000 bf16 rows of 50000 take 71 us, gated 110; of 32768 gated 44. All arithmetic is fp32 and rounds once to the output's type.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "i8_kernels.cuh"
#include "tc_common.cuh"

namespace wr {
namespace {

// ---------------------------------------------------------------- two fp32 operations in one instruction

// These kernels are short of instruction slots before they are short of bandwidth, and sm_100a has
// packed fp32 multiply, add and multiply-add (each half rounded as the plain one).
struct f32x2 {
  uint64_t v;
};
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ f32x2 splat2(float v) { return pack2(v, v); }
// A thread's vector: 8 elements as 4 pairs.
struct Vec8 {
  f32x2 p[4];
};

// ---------------------------------------------------------------- loads and stores of 8 elements

// Eight elements as loaded: 32 bytes of fp32, 16 of a 16-bit type. Loads are issued for all operands of a
// row before the first is converted, so they are kept raw. The size is a template parameter (a raw
// vector has to stay in registers), bf16 or fp16 is decided when it is converted.
template <bool F32>
struct Raw8 {
  uint32_t r[F32 ? 8 : 4];
};

__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Where element j of vector i of thread t sits in its row. VEC: 8 neighbours; otherwise (rows that
// do not start on 16 bytes) neighbouring threads take neighbouring elements, one load each.
template <bool VEC>
__device__ __forceinline__ int elem(int i, int j, int T, int t) {
  return VEC ? (i * T + t) * 8 + j : (i * 8 + j) * T + t;
}

// Vector i of thread t; zero past the row's D elements.
template <bool F32, bool VEC>
__device__ __forceinline__ Raw8<F32> load8(const uint8_t* row, int i, int T, int t, int D) {
  Raw8<F32> v;
  const int e0 = elem<VEC>(i, 0, T, t);
  if (VEC && e0 + 8 <= D) {
    const uint8_t* p = row + (int64_t)e0 * (F32 ? 4 : 2);
    const uint4 a = ld16(p);
    v.r[0] = a.x; v.r[1] = a.y; v.r[2] = a.z; v.r[3] = a.w;
    if constexpr (F32) {
      const uint4 b = ld16(p + 16);
      v.r[4] = b.x; v.r[5] = b.y; v.r[6] = b.z; v.r[7] = b.w;
    }
    return v;
  }
#pragma unroll
  for (int j = 0; j < (F32 ? 8 : 4); ++j) v.r[j] = 0;
  if (e0 >= D) return v;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = elem<VEC>(i, j, T, t);
    if (e < D) {
      if constexpr (F32) v.r[j] = reinterpret_cast<const uint32_t*>(row)[e];
      else v.r[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[e] << (16 * (j & 1));
    }
  }
  return v;
}

template <bool F32>
__device__ __forceinline__ Vec8 to_float8(const Raw8<F32>& v, int type) {
  Vec8 f;
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.p[j] = pack2(__uint_as_float(v.r[2 * j]), __uint_as_float(v.r[2 * j + 1]));
  } else if (type == WR_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.p[j] = pack2(__uint_as_float(v.r[j] << 16), __uint_as_float(v.r[j] & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&v.r[j]));
      f.p[j] = pack2(h.x, h.y);
    }
  }
  return f;
}
// The same where the type's size is not a template parameter.
template <bool VEC>
__device__ __forceinline__ Vec8 load_float8(const void* row, int type, int i, int T, int t, int D) {
  const uint8_t* p = static_cast<const uint8_t*>(row);
  return type == WR_F32 ? to_float8(load8<true, VEC>(p, i, T, t, D), type) : to_float8(load8<false, VEC>(p, i, T, t, D), type);
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
__device__ __forceinline__ void store8(uint8_t* row, int type, int i, int T, int t, int D, const Vec8& v) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack2(v.p[j], f[2 * j], f[2 * j + 1]);
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

// Every warp leaves its value in buf and every warp reduces all of them: one barrier for each
// reduction (each has its own buf). The sum is a tree, the same in every thread and every run: a row's squares
// pass through at most 4 VPT + 1 + 5 + 5 roundings. (The warps' sums one after the other: 31 roundings in place of
// the last 5, 23.8 * 2^-24 off for a row made to show it; 8192 rows of 2560 41.8 us instead of 40.2, 1000 rows of
// 32768 140 instead of 122.)
__device__ __forceinline__ float row_sum(f32x2 v2, float* buf) {
  float v, hi;
  unpack2(v2, v, hi);
  v += hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < nw ? buf[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Largest magnitude, by its bits: an infinity is above every number and a NaN above that.
__device__ __forceinline__ uint32_t row_max(float amax, uint32_t* buf) {
  uint32_t v = __float_as_uint(amax) & 0x7FFFFFFFu;
  v = __reduce_max_sync(0xffffffffu, v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < nw ? buf[threadIdx.x & 31] : 0u);
}
// max(a, |v|), NaN if either is.
__device__ __forceinline__ float max_abs(float a, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(v)));
  return r;
}
__device__ __forceinline__ float max_abs8(float a, const Vec8& v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    unpack2(v.p[j], lo, hi);
    a = max_abs(max_abs(a, lo), hi);
  }
  return a;
}

// ---------------------------------------------------------------- the 8-bit rounding

// Codes of one row with largest magnitude A: the integer nearest to 127 v / A, a tie to the even one,
// decided on the exact quotient. t = v * fl(127 / A) is off by at most 127 * 2^-23 < 1.6e-5 (two
// roundings of at most 2^-24 relative each), so only a value that close to the middle of two codes
// needs more. There the sign of 127 v - (k + 1/2) A decides, k = floor(t): both products are taken as a
// rounded part and its exact rest (31 and 32 bits: the rests have at most 8), the rounded parts are
// close enough to subtract exactly, and so are the rests. 16-bit inputs have such values in every
// third warp (v = A / 2 is one); with an fp64 division instead the quantizer of 9728 x 2560 bf16
// values took 46.5 us instead of 31.3.
// A = 0: codes 0 and scale 0. A not finite (an infinity or NaN in the row): codes 0 and scale NaN, so
// that whatever is computed from the row is NaN. Where A is so small or large that 127 / A, 127 v or a
// rest leaves the fp32 range (`wide`), the quotient is formed in fp64: 127 v and a tie's quotient are
// exact there, and any other quotient is at least 2^-40 (relative) away from a tie.
struct RowCode {
  float A, inv, scale;
  bool wide;
};
__device__ __forceinline__ RowCode row_code(uint32_t amax_bits) {
  RowCode c;
  c.A = __uint_as_float(amax_bits);
  const bool finite = amax_bits < 0x7F800000u;
  c.wide = finite && c.A > 0.f && (c.A < 0x1p-100f || c.A > 0x1p+120f);
  c.inv = finite && c.A > 0.f && !c.wide ? __fdiv_rn(127.f, c.A) : 0.f;
  c.scale = finite ? __fdiv_rn(c.A, 127.f) : __uint_as_float(0x7FC00000u);
  if (!finite) c.A = 0.f;
  return c;
}
__device__ __noinline__ float code_exact(float v, float A) { return (float)rint((double)v * 127.0 / (double)A); }
// The codes of 8 values, a byte each. Adding 1.5 * 2^23 rounds t to the nearest integer (ties to even)
// and leaves it, as two's complement, in the low bits.
__device__ __forceinline__ void codes8(const RowCode& c, const Vec8& v, uint32_t p[2]) {
  constexpr float kMagic = 12582912.f;
  if (c.A == 0.f) {
    p[0] = p[1] = 0;
    return;
  }
  const f32x2 inv = splat2(c.inv), magic = splat2(kMagic), unmagic = splat2(-kMagic), minus = splat2(-1.f);
  float r[8], far = 0.f;   // far: the largest distance from a code, of 1/2 at most
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 t = mul2(v.p[j], inv), rr = add2(t, magic);
    const f32x2 d = fma2(t, minus, add2(rr, unmagic));
    unpack2(rr, r[2 * j], r[2 * j + 1]);
    float lo, hi;
    unpack2(d, lo, hi);
    far = fmaxf(fmaxf(far, fabsf(lo)), fabsf(hi));
  }
  if (far > 0.49998f || c.wide) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(v.p[j], f[2 * j], f[2 * j + 1]);
    if (c.wide) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = code_exact(f[j], c.A) + kMagic;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float k = floorf(__fmul_rn(f[j], c.inv)), h = k + 0.5f;
        const float v1 = __fmul_rn(127.f, f[j]), v0 = __fmaf_rn(127.f, f[j], -v1);
        const float a1 = __fmul_rn(h, c.A), a0 = __fmaf_rn(h, c.A, -a1);
        const float d = __fadd_rn(__fsub_rn(v1, a1), __fsub_rn(v0, a0));
        // a tie: k or k + 1, whichever is even (kMagic + h rounds to even)
        r[j] = d > 0.f ? k + 1.f + kMagic : d < 0.f ? k + kMagic : h + kMagic;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __byte_perm(__float_as_uint(r[4 * h]), __float_as_uint(r[4 * h + 1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(r[4 * h + 2]), __float_as_uint(r[4 * h + 3]), 0x0040);
    p[h] = __byte_perm(lo, hi, 0x5410);
  }
}

template <bool VEC>
__device__ __forceinline__ void store_codes8(int8_t* row, int i, int T, int t, int D, const RowCode& c, const Vec8& v) {
  uint32_t p[2];
  codes8(c, v, p);
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

// silu(g) x = g x / (1 + 2^t), t = -g log2 e, off by less than 10 * 2^-24 for every gate from -87.3 on: log2 e has two
// parts, so that what t loses when it is rounded, and what the first part lacks (1.3e-8 |g| of the result: 19 * 2^-24
// at g = -86), come back as a first-order term, 2^(t + r) = 2^t (1 + r ln 2). 2^t is off by at most 2^-22 and the
// reciprocal by 2^-23 (the approximate instructions); the factor, the sum and two products round once each. t is held
// below 126 so that an overflow cannot meet a zero: there silu is below 1.1e-36 and reads as 0. g is held below 128
// where it enters the exponent, so that t stays finite for every finite g (2^t is 0 there, and silu(g) = g).
__device__ __forceinline__ Vec8 silu_mul(const Vec8& g, const Vec8& x) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500011e-8f;   // log2 e
  const f32x2 hi2 = splat2(kHi), minus_hi = splat2(-kHi), lo2 = splat2(kLo), minus_ln2 = splat2(-0.6931471805599453f);
  const f32x2 one = splat2(1.f);
  Vec8 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi, elo, ehi;
    unpack2(g.p[j], lo, hi);
    const f32x2 held = pack2(fminf(lo, 128.f), fminf(hi, 128.f));
    unpack2(mul2(held, minus_hi), lo, hi);
    lo = fminf(lo, 126.f);
    hi = fminf(hi, 126.f);
    const f32x2 minus_r = fma2(held, lo2, fma2(held, hi2, pack2(lo, hi)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(elo) : "f"(lo));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ehi) : "f"(hi));
    const f32x2 s = fma2(pack2(elo, ehi), fma2(minus_r, minus_ln2, one), one);
    unpack2(s, lo, hi);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(elo) : "f"(lo));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ehi) : "f"(hi));
    o.p[j] = mul2(mul2(g.p[j], pack2(elo, ehi)), x.p[j]);
  }
  return o;
}

__host__ __device__ inline int type_bytes(int type) { return type == WR_F32 ? 4 : (type == WR_I8 ? 1 : 2); }

// ---------------------------------------------------------------- row quantizer

// VPT > 0: the row stays in registers. VPT = 0: rows longer than that; read twice (the second time
// mostly from L2), in steps of one vector a thread.
template <int VPT, int MAXT, bool VEC, bool F32, bool GATED>
__global__ void __launch_bounds__(MAXT) quantize_rows_kernel(const QuantRowsArgs a) {
  __shared__ uint32_t buf[32];
  const int T = blockDim.x, t = threadIdx.x;
  const int64_t m = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  tc::grid_launch_dependents();   // a product that follows may set itself up meanwhile
  if (m >= a.M) return;   // (whole warps)
  constexpr int es = F32 ? 4 : 2;
  const uint8_t* x = a.x + m * a.ldx * es;
  const uint8_t* g = GATED ? a.gate + m * a.ldg * es : nullptr;
  int8_t* q = a.q + m * a.ldq;
  float amax = 0.f;
  if constexpr (VPT > 0) {
    Raw8<F32> rx[VPT], rg[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      rx[i] = load8<F32, VEC>(x, i, T, t, a.K);
      if (GATED) rg[i] = load8<F32, VEC>(g, i, T, t, a.K);
    }
    Vec8 v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      v[i] = to_float8(rx[i], a.type);
      if (GATED) v[i] = silu_mul(to_float8(rg[i], a.type), v[i]);
      amax = max_abs8(amax, v[i]);
    }
    const RowCode c = row_code(row_max(amax, buf));
#pragma unroll
    for (int i = 0; i < VPT; ++i) store_codes8<VEC>(q, i, T, t, a.K, c, v[i]);
    if (t == 0) a.scale[m] = c.scale;
  } else {
    const int steps = (a.K + 8 * T - 1) / (8 * T);
    auto step = [&](int i) {
      const Raw8<F32> rx = load8<F32, VEC>(x, i, T, t, a.K);
      if (!GATED) return to_float8(rx, a.type);
      return silu_mul(to_float8(load8<F32, VEC>(g, i, T, t, a.K), a.type), to_float8(rx, a.type));
    };
#pragma unroll 2
    for (int i = 0; i < steps; ++i) amax = max_abs8(amax, step(i));
    const RowCode c = row_code(row_max(amax, buf));
    for (int i = 0; i < steps; ++i) store_codes8<VEC>(q, i, T, t, a.K, c, step(i));
    if (t == 0) a.scale[m] = c.scale;
  }
}

// ---------------------------------------------------------------- residual + norm

template <int VPT>
__device__ __forceinline__ f32x2 squares(const Vec8 (&v)[VPT], f32x2 scale) {
  f32x2 ss = splat2(0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x2 x = mul2(v[i].p[j], scale);
      ss = fma2(x, x, ss);
    }
  return ss;
}
// 1 / sqrt(mean of squares + eps) of a row. Where the sum leaves fp32's range (values beyond 2^56, or below
// 2^-50 with nothing to speak of added) the squares are summed again of values scaled by a power of two: a
// row of numbers of that size is normed like any other.
template <int VPT>
__device__ __forceinline__ float inv_rms(const Vec8 (&v)[VPT], float inv_d, float eps, float* buf, float* buf2) {
  f32x2 s2 = splat2(0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s2 = fma2(v[i].p[j], v[i].p[j], s2);
  const float ss = row_sum(s2, buf);
  if (ss <= 3.4e38f && (ss >= 1e-30f || eps >= 1e-30f)) return rsqrtf(ss * inv_d + eps);
  const float s = ss < 1.f ? 0x1p+80f : 0x1p-80f;
  return s * rsqrtf(row_sum(squares(v, splat2(s)), buf2) * inv_d + eps * s * s);
}

// B32, R32, W32: whether the block, the residual, and the weights (the gate is usually like them) are fp32.
struct NormArgs {
  wr_residual_norm_args p;
  float inv_d;           // 1 / D
};

template <int VPT, int MAXT, bool VEC, bool B32, bool R32, bool W32>
__global__ void __launch_bounds__(MAXT) residual_norm_kernel(const NormArgs na) {
  const wr_residual_norm_args& a = na.p;
  __shared__ float buf_post[32], buf_norm[32];
  __shared__ float wide_post[32], wide_norm[32];
  __shared__ uint32_t buf_max[32];
  const int T = blockDim.x, t = threadIdx.x, D = (int)a.D;
  const int64_t m = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  tc::grid_launch_dependents();   // a product that follows may set itself up meanwhile
  if (m >= a.M) return;   // (whole warps)
  const uint8_t* b = static_cast<const uint8_t*>(a.block) + m * a.ld_block * (B32 ? 4 : 2);
  const uint8_t* h = static_cast<const uint8_t*>(a.residual) + m * a.ld_residual * (R32 ? 4 : 2);
  const uint8_t* g = static_cast<const uint8_t*>(a.gate) + m * a.ld_gate * type_bytes(a.gate_type);
  const bool g_early = a.gate && (a.gate_type == WR_F32) == W32;   // else (rare) it is loaded when it is used
  const uint8_t* pw = static_cast<const uint8_t*>(a.post_weight);
  const uint8_t* nw = static_cast<const uint8_t*>(a.norm_weight);
  // everything the row needs before its last reduction is loaded at once; the last weights while that runs
  Raw8<B32> rb[VPT];
  Raw8<R32> rh[VPT];
  Raw8<W32> rp[VPT], rg[VPT], rn[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (a.block) rb[i] = load8<B32, VEC>(b, i, T, t, D);
    if (a.residual) rh[i] = load8<R32, VEC>(h, i, T, t, D);
    if (g_early) rg[i] = load8<W32, VEC>(g, i, T, t, D);
    if (pw) rp[i] = load8<W32, VEC>(pw, i, T, t, D);
  }
  const f32x2 offset = splat2(a.weight_offset), rs = splat2(a.residual_scale);
  auto scale8 = [&](Vec8& x, float r, const uint8_t* weight, const Raw8<W32>& rw) {
    const f32x2 rr = splat2(r);
    if (weight) {
      const Vec8 w = to_float8(rw, a.weight_type);
#pragma unroll
      for (int j = 0; j < 4; ++j) x.p[j] = mul2(mul2(x.p[j], rr), add2(w.p[j], offset));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x.p[j] = mul2(x.p[j], rr);
    }
  };
  // elements past the row are zero in every operand and stay so
  Vec8 v[VPT];   // the block's output, then h'
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (a.block) v[i] = to_float8(rb[i], a.block_type);
    else
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].p[j] = splat2(0.f);
  }
  if (a.post_norm) {
    const float r = inv_rms<VPT>(v, na.inv_d, a.eps, buf_post, wide_post);
#pragma unroll
    for (int i = 0; i < VPT; ++i) scale8(v[i], r, pw, rp[i]);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (a.gate) {
      const Vec8 w = g_early ? to_float8(rg[i], a.gate_type) : load_float8<VEC>(g, a.gate_type, i, T, t, D);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].p[j] = mul2(v[i].p[j], w.p[j]);
    }
    if (a.residual) {
      const Vec8 w = to_float8(rh[i], a.residual_type);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].p[j] = fma2(rs, w.p[j], v[i].p[j]);
    }
    if (nw) rn[i] = load8<W32, VEC>(nw, i, T, t, D);
  }
  if (a.residual_out) {
    uint8_t* o = static_cast<uint8_t*>(a.residual_out) + m * a.ld_residual_out * (R32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < VPT; ++i) store8<VEC>(o, a.residual_type, i, T, t, D, v[i]);
  }
  if (!a.y) return;
  const float r = inv_rms<VPT>(v, na.inv_d, a.eps, buf_norm, wide_norm);
  uint8_t* y = static_cast<uint8_t*>(a.y) + m * a.ld_y * type_bytes(a.y_type);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    scale8(v[i], r, nw, rn[i]);
    // (a row with r = infinity or NaN is NaN in all its elements; past its end 0 r is NaN too)
    if (a.y_type == WR_I8) amax = max_abs8(amax, v[i]);
    else store8<VEC>(y, a.y_type, i, T, t, D, v[i]);
  }
  if (a.y_type == WR_I8) {
    const RowCode c = row_code(row_max(amax, buf_max));
#pragma unroll
    for (int i = 0; i < VPT; ++i) store_codes8<VEC>(reinterpret_cast<int8_t*>(y), i, T, t, D, c, v[i]);
    if (t == 0) a.y_scale[m] = c.scale;
  }
}

inline bool rows_aligned(int64_t M, int64_t ld, int bytes) { return M == 1 || ld * bytes % 16 == 0; }

// Threads that hold a row of D elements, VPT vectors of 8 each.
inline int row_threads(int64_t D, int vpt) { return (int)std::min<int64_t>(1024, ((D + 8 * vpt - 1) / (8 * vpt) + 31) / 32 * 32); }

// Vectors a thread. Few rows: one or two, the shortest way through a row (one gated row of 9728 fp32 values:
// 3.5 us with two, 3.9 with four). Many: two, since a thread's work in the
// reductions is the same for 16 elements as for 8 and instructions run out before bandwidth does, while
// four leave too few warps to hide the loads (8192 rows of 2560, fp32 block, bf16 residual, a gate: 46.6, 40.5
// and 58.7 us with one, two and four; 500 rows: 5.1, 5.2 and 6.4). Four where two would make a CTA of more
// than `most` threads: the quantizer holds less and gains from four earlier (2000 gated rows of 8192 bf16:
// 19.0 against 22.2 us; the norm: 39.7 against 33.2).
constexpr int64_t kManyRows = 2 * 148;
inline int row_vpt(int64_t M, int64_t D, int most) {
  const int64_t vecs = (D + 7) / 8;
  if (M < kManyRows) return vecs <= 512 ? 1 : vecs <= 2048 ? 2 : 4;
  return vecs <= 32 ? 1 : vecs <= 2 * most ? 2 : 4;
}
// The launch: a CTA for each row, or, where a warp holds a row, four rows a CTA.
struct RowGrid {
  dim3 grid, block;
  RowGrid(int64_t M, int T) {
    const unsigned rows = T == 32 && M >= kManyRows ? 4 : 1;
    grid = dim3((unsigned)((M + rows - 1) / rows));
    block = dim3((unsigned)T, rows);
  }
};

template <int VPT, int MAXT, bool VEC>
cudaError_t run_quantize(const QuantRowsArgs& a, cudaStream_t stream) {
  const RowGrid d(a.M, row_threads(a.K, VPT > 0 ? VPT : 4));
  if (a.type == WR_F32) {
    return launch_plain(a.gate ? quantize_rows_kernel<VPT, MAXT, VEC, true, true> : quantize_rows_kernel<VPT, MAXT, VEC, true, false>,
                        d.grid, d.block, stream, a);
  }
  return launch_plain(a.gate ? quantize_rows_kernel<VPT, MAXT, VEC, false, true> : quantize_rows_kernel<VPT, MAXT, VEC, false, false>,
                      d.grid, d.block, stream, a);
}
template <bool VEC>
cudaError_t run_quantize(const QuantRowsArgs& a, cudaStream_t stream) {
  const int vpt = row_vpt(a.M, a.K, 256);
  if (a.K > 32768) return run_quantize<0, 1024, VEC>(a, stream);
  if (a.K > 16384) return run_quantize<4, 1024, VEC>(a, stream);
  if (vpt == 1) return run_quantize<1, 512, VEC>(a, stream);
  if (vpt == 2) return a.K <= 8192 ? run_quantize<2, 512, VEC>(a, stream) : run_quantize<2, 1024, VEC>(a, stream);
  return run_quantize<4, 512, VEC>(a, stream);
}

template <int VPT, int MAXT, bool VEC, bool B32, bool R32>
cudaError_t run_norm(const NormArgs& a, bool w32, cudaStream_t stream) {
  const RowGrid d(a.p.M, row_threads(a.p.D, VPT));
  return launch_plain(w32 ? residual_norm_kernel<VPT, MAXT, VEC, B32, R32, true> : residual_norm_kernel<VPT, MAXT, VEC, B32, R32, false>,
                      d.grid, d.block, stream, a);
}
template <int VPT, int MAXT, bool VEC>
cudaError_t run_norm(const NormArgs& a, bool w32, cudaStream_t stream) {
  const bool b32 = a.p.block_type == WR_F32, r32 = a.p.residual_type == WR_F32;
  if (b32 && r32) return run_norm<VPT, MAXT, VEC, true, true>(a, w32, stream);
  else if (b32) return run_norm<VPT, MAXT, VEC, true, false>(a, w32, stream);
  else if (r32) return run_norm<VPT, MAXT, VEC, false, true>(a, w32, stream);
  else return run_norm<VPT, MAXT, VEC, false, false>(a, w32, stream);
}
template <bool VEC>
cudaError_t run_norm(const NormArgs& a, bool w32, cudaStream_t stream) {
  const int vpt = row_vpt(a.p.M, a.p.D, 512);
  if (a.p.D > 16384) return run_norm<4, 1024, VEC>(a, w32, stream);
  if (vpt == 1) return run_norm<1, 512, VEC>(a, w32, stream);
  if (vpt == 2) return a.p.D <= 8192 ? run_norm<2, 512, VEC>(a, w32, stream) : run_norm<2, 1024, VEC>(a, w32, stream);
  return run_norm<4, 512, VEC>(a, w32, stream);
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantRowsArgs& a, cudaStream_t stream) {
  const int es = type_bytes(a.type);
  const bool vec = rows_aligned(a.M, a.ldx, es) && (!a.gate || rows_aligned(a.M, a.ldg, es)) && (a.M == 1 || a.ldq % 8 == 0);
  return vec ? run_quantize<true>(a, stream) : run_quantize<false>(a, stream);
}

cudaError_t launch_residual_norm(const wr_residual_norm_args& a, cudaStream_t stream) {
  const bool vec = (!a.block || rows_aligned(a.M, a.ld_block, type_bytes(a.block_type))) &&
                   (!a.residual || rows_aligned(a.M, a.ld_residual, type_bytes(a.residual_type))) &&
                   (!a.residual_out || rows_aligned(a.M, a.ld_residual_out, type_bytes(a.residual_type))) &&
                   (!a.gate || rows_aligned(a.M, a.ld_gate, type_bytes(a.gate_type))) &&
                   (!a.y || (a.y_type == WR_I8 ? a.M == 1 || a.ld_y % 8 == 0 : rows_aligned(a.M, a.ld_y, type_bytes(a.y_type))));
  NormArgs na{a, (float)(1.0 / (double)a.D)};
  const bool w32 = a.post_weight || a.norm_weight ? a.weight_type == WR_F32 : a.gate_type == WR_F32;
  return vec ? run_norm<true>(na, w32, stream) : run_norm<false>(na, w32, stream);
}

}  // namespace wr
