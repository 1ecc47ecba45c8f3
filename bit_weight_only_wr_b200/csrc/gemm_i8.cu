// Int8 product with a scale for each token and each output channel (sm_100a):
//   y[m,n] = (sum_k x[m,k] w[n,k]) x_scale[m] w_scale[n] + bias[n]
// The sums are exact 32-bit integers (K <= 131071), so that they do not depend on the order or on how
// K is split; the conversion and the two products are fp32, in this order, in every kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "i8_kernels.cuh"
#include "tc_common.cuh"
#include "tc_kernels.cuh"

namespace wr {
namespace {

using namespace tc;

// The steps from a sum to y, each rounded (the intrinsics are never joined to a multiply-add): every form ends in
// these two, so that y has the same bits in all of them.
__device__ __forceinline__ float scaled(int acc, float xs, float ws) { return __fmul_rn(__fmul_rn(__int2float_rn(acc), xs), ws); }
__device__ __forceinline__ float biased(float v, float bias) { return __fadd_rn(v, bias); }
__device__ __forceinline__ float finished(int acc, float xs, float ws, const float* bias, int n) {
  const float v = scaled(acc, xs, ws);
  return bias ? biased(v, bias[n]) : v;
}
__device__ __forceinline__ void store_y(void* y, int type, int64_t at, float v) {
  if (type == WR_F32) static_cast<float*>(y)[at] = v;
  else if (type == WR_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// ---------------------------------------------------------------- one or two tokens: dp4a, one pass over w

// 16 bytes, or zeros (no load) where !in; KEEP: in L1 too. (None of these kernels reads through the read-only
// path: they may start before the kernel that writes their inputs has ended, see launch_overlapped.)
template <bool KEEP>
__device__ __forceinline__ uint4 chunk_if(const int8_t* p, bool in) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (KEEP)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "l"(p), "r"((int)in));
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n @p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "l"(p), "r"((int)in));
  return v;
}
// The last `n` < 16 bytes of a row (p 16-byte aligned), then zeros: whole words, then single bytes.
__device__ __forceinline__ uint4 row_end(const int8_t* p, int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = 4 * i + 4 <= n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
  uint32_t rest = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if ((n & ~3) + i < n) rest |= (uint32_t)(uint8_t)p[(n & ~3) + i] << (8 * i);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i == n / 4) w[i] = rest;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int acc) {
  acc = __dp4a((int)a.x, (int)b.x, acc);
  acc = __dp4a((int)a.y, (int)b.y, acc);
  acc = __dp4a((int)a.z, (int)b.z, acc);
  return __dp4a((int)a.w, (int)b.w, acc);
}

// `share` warps (1, 2 or 4) of a CTA share a row of w and read it once, 512 bytes a warp and step with eight
// steps in flight; x comes from L1. Memory latency is what a matrix of this size is bound by, so share is
// what lets a warp have all of its bytes on their way at once (up to K = 16384). Where there are rows for more
// than two rounds of CTAs, a CTA takes rows in turn: 21312 rows of 2064 bytes 8.8 us, a CTA for every four rows 9.7;
// 40000 of 2560 with two tokens 18.8 and 19.9, with one 17.2 and 17.0; of 9728 66 and 64. In two rounds and fewer the
// two differ either way (7992 rows of 4096: 7.3 and 6.7, 10656 rows of 2560: 5.6 and 6.1).
constexpr int kGemvThreads = 128, kGemvCtas = 148 * 9;   // nine CTAs fill an SM's registers
template <int MT>
__global__ void __launch_bounds__(kGemvThreads, 9) gemv_i8_kernel(const GemmI8Args a, const int share) {
  __shared__ int parts[2][kGemvThreads / 32][MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = kGemvThreads / 32 / share, part = warp % share;
  const int whole = a.K / 16, rest = a.K % 16;   // 16-byte pieces of a row
  int n = blockIdx.x * rows + warp / share;
  grid_launch_dependents();
  // the first row may come to L2 while the kernel before this one still runs
  if (n < a.N)
    for (int k = (part * 32 + lane) * 128; k < a.K; k += share * 4096) prefetch_l2(a.w + (int64_t)n * a.ldw + k);
  grid_dependency_wait();
  const float xs = a.x_scale[min(lane, MT - 1)];
  for (int first = blockIdx.x * rows, par = 0; first < a.N; first += gridDim.x * rows, n += gridDim.x * rows, par ^= 1) {
    const bool real = n < a.N;
    const int8_t* w = a.w + (int64_t)(real ? n : 0) * a.ldw;
    const float ws = real ? a.w_scale[n] : 0.f;
    int acc[MT] = {};
    if (rest != 0 && part == 0 && lane == 0) {
      const uint4 wv = row_end(w + 16 * whole, rest);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = dot16(wv, row_end(a.x + m * a.ldx + 16 * whole, rest), acc[m]);
    }
    constexpr int U = 8;
    for (int base = part * 32; base < whole; base += 32 * share * U) {
      uint4 wv[U], xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = base + 32 * share * u + lane;
        wv[u] = chunk_if<false>(w + 16 * c, c < whole);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = base + 32 * share * u + lane;
          xv[u] = chunk_if<true>(a.x + m * a.ldx + 16 * c, c < whole);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) acc[m] = dot16(wv[u], xv[u], acc[m]);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = __reduce_add_sync(0xffffffffu, acc[m]);
    if (share > 1) {
      if (lane == 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m) parts[par][warp][m] = acc[m];
      }
      __syncthreads();   // (the other buffer was read before this barrier and is written after it)
      if (part == 0) {
        for (int i = 1; i < share; ++i) {
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m] += parts[par][warp + i][m];
        }
      }
    }
    if (lane < MT && part == 0 && real) {
      int sum = acc[0];
#pragma unroll
      for (int m = 1; m < MT; ++m) sum = lane == m ? acc[m] : sum;
      store_y(a.y, a.y_type, lane * a.ldy + n, finished(sum, xs, ws, a.bias, n));
    }
  }
}

template <int MT>
cudaError_t run_gemv(const GemmI8Args& a, cudaStream_t stream) {
  const int steps = (a.K + 511) / 512;
  const int share = steps <= 8 ? 1 : steps <= 16 ? 2 : 4, rows = kGemvThreads / 32 / share;
  const int ctas = (a.N + rows - 1) / rows, grid = ctas <= 2 * kGemvCtas ? ctas : kGemvCtas;
  return launch_overlapped(gemv_i8_kernel<MT>, dim3((unsigned)grid), dim3(kGemvThreads), 0, 1, stream, a, share);
}

// ---------------------------------------------------------------- up to 16 tokens: mma.sync, one pass over w

// Few tokens are bound by the latency of the rows, not by products, and a tile on tcgen05 has a start and an end
// of 2 us. Here a CTA owns 16 rows of w (the m of mma.m16n8k32) and NT times 8 tokens (its n); its eight warps
// take turns of 128 bytes of K, U turns at once, and add up in shared memory. The order of K inside an MMA is
// free as long as both operands keep it: lane 4 g + t loads 32 contiguous bytes of rows g and g + 8 and of
// tokens g, g + 8, so that rows come in whole 128-byte lines straight into the registers that the MMAs take.
// 8 tokens of 2560 x 4096 3.9 us (tcgen05 5.2), 4096 x 2560 3.3 (4.9), 6144 x 2560 4.0 (6.2); the last bytes of
// rows stand outside the loop (inside it: 4.5, 2560 x 4096). A ring of bulk copies in its place: 6.3.
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
__device__ __forceinline__ void mma_i8(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int U, int CTAS, int NT>
__global__ void __launch_bounds__(kFewThreads, CTAS) few_i8_kernel(const GemmI8Args a) {
  __shared__ int parts[kFewWarps][8 * NT][17];   // [warp][token][row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int whole = a.K / 16, rest = a.K % 16;   // 16-byte pieces of a row
  grid_launch_dependents();
  // the rows may come to L2 while the kernel before this one still runs
  {
    const int lines = (a.K + 127) / 128, row = threadIdx.x & 15;
    if (n0 + row < a.N)
      for (int l = threadIdx.x >> 4; l < lines; l += kFewThreads / 16) prefetch_l2(a.w + (int64_t)(n0 + row) * a.ldw + l * 128);
  }
  grid_dependency_wait();
  const bool real0 = n0 + g < a.N, real1 = n0 + g + 8 < a.N;
  const int8_t* w0 = a.w + (int64_t)(real0 ? n0 + g : 0) * a.ldw;
  const int8_t* w1 = a.w + (int64_t)(real1 ? n0 + g + 8 : 0) * a.ldw;
  const int8_t* x[NT];
  bool realx[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    realx[j] = g + 8 * j < a.M;
    x[j] = a.x + (int64_t)(realx[j] ? g + 8 * j : 0) * a.ldx;
  }
  int c[NT][4] = {};
  const int full = a.K / 128, steps = (a.K + 127) / 128;   // turns of 128 bytes: whole ones, all
  for (int s0 = warp; s0 < full; s0 += kFewWarps * U) {
    uint4 p0[U][2], p1[U][2], px[U][2][NT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int s = s0 + kFewWarps * u, k = s * 8 + 2 * t + h;   // 16-byte piece
        p0[u][h] = chunk_if<false>(w0 + 16 * k, s < full && real0);
        p1[u][h] = chunk_if<false>(w1 + 16 * k, s < full && real1);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int s = s0 + kFewWarps * u, k = s * 8 + 2 * t + h;
#pragma unroll
        for (int j = 0; j < NT; ++j) px[u][h][j] = chunk_if<true>(x[j] + 16 * k, s < full && realx[j]);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_i8(c[j], p0[u][h].x, p1[u][h].x, p0[u][h].y, p1[u][h].y, px[u][h][j].x, px[u][h][j].y);
          mma_i8(c[j], p0[u][h].z, p1[u][h].z, p0[u][h].w, p1[u][h].w, px[u][h][j].z, px[u][h][j].w);
        }
      }
  }
  if (full < steps && warp == full % kFewWarps) {   // the rows' last bytes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = full * 8 + 2 * t + h;
      uint4 p0 = chunk_if<false>(w0 + 16 * k, k < whole && real0), p1 = chunk_if<false>(w1 + 16 * k, k < whole && real1);
      if (rest != 0 && k == whole) {
        if (real0) p0 = row_end(w0 + 16 * k, rest);
        if (real1) p1 = row_end(w1 + 16 * k, rest);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 px = chunk_if<true>(x[j] + 16 * k, k < whole && realx[j]);
        if (rest != 0 && k == whole && realx[j]) px = row_end(x[j] + 16 * k, rest);
        mma_i8(c[j], p0.x, p1.x, p0.y, p1.y, px.x, px.y);
        mma_i8(c[j], p0.z, p1.z, p0.w, p1.w, px.z, px.w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    parts[warp][8 * j + 2 * t][g] = c[j][0];
    parts[warp][8 * j + 2 * t + 1][g] = c[j][1];
    parts[warp][8 * j + 2 * t][g + 8] = c[j][2];
    parts[warp][8 * j + 2 * t + 1][g + 8] = c[j][3];
  }
  const int n = n0 + (threadIdx.x & 15);
  const float ws = n < a.N ? a.w_scale[n] : 0.f;
  __syncthreads();
  for (int m = threadIdx.x >> 4; m < a.M; m += kFewThreads / 16) {
    if (n >= a.N) break;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kFewWarps; ++i) sum += parts[i][m][threadIdx.x & 15];
    store_y(a.y, a.y_type, m * a.ldy + n, finished(sum, a.x_scale[m], ws, a.bias, n));
  }
}

// ---------------------------------------------------------------- more tokens: tcgen05 kind::i8

// The channels are the rows of the MMA (A, 128 a CTA), the tokens its columns (B), so that a thread of the
// epilogue owns one channel and a warp writes 32 neighbouring ones. A tile is 128 channels (256 for a
// CTA pair) by tn tokens; its K is cut in blocks of 128 bytes, one stage of a ring each (TMA, 128-byte
// swizzle, zeros behind the ends of K, M and N). Warps: 0 loads (TMA), 1 issues the MMAs, 2-9 are the
// epilogue (two for each 32 TMEM lanes 32 (warp % 4) .., which take turns of 16 tokens). Every wait on an
// mbarrier is bounded, and a CTA whose wait ran out still meets the others at every barrier (see settle).
//
// CTA pairs (cta_group::2) load each operand once for 256 x tn outputs. Two forms (plan_gemm_i8 chooses
// by the time it expects of each):
//   split       a cluster of `split` CTAs, or pairs, shares a tile, each with its part of K; they leave their
//               int32 sums in shared memory and each finishes its part of the tokens from all of them.
//               (Without a cluster two CTAs fit an SM.)
//   persistent  pairs take whole tiles in turn; the epilogue of a tile overlaps the products of the next
//               (two accumulators).
constexpr int kGemmThreads = 320, kEpilogueThreads = 256;
constexpr int kMaxStages = 12;

struct GemmBars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
  uint32_t copies, mmas, accs;   // how far the roles got: stages filled, stages multiplied, accumulators committed
};

struct GemmParams {
  GemmI8Args a;
  int tn, mt, kb, split, stages, tmem_cols;
  int whole, cut, cut_tn, units;   // persistent form: see unit_of
  int* err;
  uint64_t wait_ns;   // limit of a wait (0: gives up at its second look)
};

__device__ __forceinline__ void init_bars(GemmBars& bars, int stages, int empties) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], empties);
    }
    bars.abort_flag = 0;
    bars.copies = bars.mmas = bars.accs = 0;
    fence_barrier_init();
  }
}

// Position in the ring of stages.
struct Ring {
  int s = 0;
  uint32_t ph = 0, count = 0;
  __device__ __forceinline__ void next(int stages) {
    ++count;
    if (++s == stages) {
      s = 0;
      ph ^= 1;
    }
  }
};

// mbar_wait of a whole warp, which goes on or gives up as one: the lanes decide together. (A vote after every wait in
// its place: 32 tokens of 6144 x 2560 6.1 -> 6.4 us.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, GemmBars& bars, const GemmParams& p, int code) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  volatile int* abort_flag = &bars.abort_flag;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15u) == 0 || p.wait_ns == 0) {
      const uint32_t here = __activemask();
      if (__any_sync(here, *abort_flag != 0)) return false;
      if (__any_sync(here, global_ns() - t0 >= p.wait_ns)) break;
    }
  }
  *abort_flag = 1;
  if (p.err) atomicCAS(p.err, 0, code);
  return false;
}

// The barrier and parity of the last stage that the loading thread filled. It leaves when that has been multiplied, and
// with it (commits arrive in order) all of them: no arrival is then under way to this CTA's barriers.
__device__ __forceinline__ uint64_t* last_empty(GemmBars& bars, const Ring& r, int stages, uint32_t& parity) {
  parity = r.s == 0 ? r.ph ^ 1 : r.ph;
  return &bars.empty[r.s == 0 ? stages - 1 : r.s - 1];
}

// A wait that ran out raises its CTA's flag; before a cluster meets, every warp passes the flag on, so that all of
// its CTAs leave the same way.
__device__ __forceinline__ void pass_on_abort(GemmBars& bars, int size, int lane) {
  __syncwarp();
  if (*(volatile int*)&bars.abort_flag && lane < size) st_cluster_u32(cluster_addr(&bars.abort_flag, lane), 1);
}

// On the way out of an aborted cluster, after all of its warps have met: the copies in flight land and the MMAs
// issued end (bounded waits) before shared and tensor memory are given up. The CTAs of a pair share the leader's
// `full` barriers and stop independently: what one of them loaded without the other is made up for on the barrier.
// A CTA loads `bytes` into a stage, cut_bytes from stage cut_from on.
template <bool PAIR>
__device__ __noinline__ void settle(GemmBars* bars, uint32_t stages, uint32_t leader, uint32_t bytes, uint32_t cut_bytes,
                                    uint32_t cut_from) {
  const bool leads = !PAIR || cluster_rank() == leader;
  if (threadIdx.x == 0 && leads) {
    const uint32_t mine = bars->copies, theirs = PAIR ? ld_cluster_u32(cluster_addr(&bars->copies, leader + 1)) : mine;
    const uint32_t most = max(mine, theirs);
    for (uint32_t j = most > stages ? most - stages : 0; j < most; ++j) {
      uint64_t* bar = &bars->full[j % stages];
      if (j >= mine) mbar_arrive_expect_tx(bar, j >= cut_from ? cut_bytes : bytes);
      else if (j >= theirs) mbar_complete_tx(bar, j >= cut_from ? cut_bytes : bytes);
      if (!mbar_wait_drain(bar, (j / stages) & 1)) break;
    }
  }
  if (threadIdx.x == 32) {   // (the commits arrive in both CTAs of a pair)
    const uint32_t mmas = PAIR ? ld_cluster_u32(cluster_addr(&bars->mmas, leader)) : bars->mmas;
    const uint32_t accs = PAIR ? ld_cluster_u32(cluster_addr(&bars->accs, leader)) : bars->accs;
    if (mmas > 0) mbar_wait_drain(&bars->empty[(mmas - 1) % stages], ((mmas - 1) / stages) & 1);
    if (accs > 0) mbar_wait_drain(&bars->acc_full[(accs - 1) & 1], ((accs - 1) >> 1) & 1);
  }
}

// y's 16-bit types: one value, and two neighbouring channels.
struct Bf16Out {
  static __device__ __forceinline__ uint16_t one(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
  static __device__ __forceinline__ uint32_t two(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
struct F16Out {
  static __device__ __forceinline__ uint16_t one(float v) { return __half_as_ushort(__float2half_rn(v)); }
  static __device__ __forceinline__ uint32_t two(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// store16 of a 16-bit y: neighbouring lanes exchange values, so that even lanes store pairs of channels of the even
// tokens and odd lanes those of the odd ones (half the stores and conversions; needs rows that start on 4 bytes).
template <typename Out>
__device__ __forceinline__ void store16_half(const GemmI8Args& a, int m, int left, int ch, int lane, const float v[16]) {
  uint16_t* y = static_cast<uint16_t*>(a.y) + (int64_t)m * a.ldy + ch;
  const bool odd = lane & 1;
  if ((a.ldy & 1) == 0 && (ch - lane) + 32 <= a.N && left >= 16) {
    // the warp's 32 channels are all real: lane pairs cover them
    uint32_t* y2 = reinterpret_cast<uint32_t*>(y - odd) + (odd ? a.ldy / 2 : 0);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
      y2[(i / 2) * a.ldy] = Out::two(odd ? got : v[i], odd ? v[i + 1] : got);
    }
    return;
  }
  if (ch >= a.N) return;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < left) y[i * a.ldy] = Out::one(v[i]);
}

// Writes this thread's channel of 16 tokens from token m on (`left` of them real): v plus the bias. A
// warp holds 32 neighbouring channels, so a token's store is 128 contiguous bytes of fp32.
__device__ __forceinline__ void store16(const GemmI8Args& a, int m, int left, int ch, int lane, float v[16], float bias) {
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = biased(v[i], bias);
  }
  if (a.y_type == WR_BF16) return store16_half<Bf16Out>(a, m, left, ch, lane, v);
  if (a.y_type == WR_F16) return store16_half<F16Out>(a, m, left, ch, lane, v);
  if (ch >= a.N) return;
  float* y = static_cast<float*>(a.y) + (int64_t)m * a.ldy + ch;
  if (left >= 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i * a.ldy] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) y[i * a.ldy] = v[i];
  }
}

// 16 tokens of one channel from their sums. xs: their scales (shared memory, readable past `left`).
__device__ __forceinline__ void finish16(const GemmI8Args& a, const int sum[16], const float* xs, int m, int left, int ch, int lane, float ws,
                                         float bias) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = scaled(sum[i], xs[i], ws);
  store16(a, m, left, ch, lane, v, bias);
}

// The scales of a tile's tokens, to shared memory, by the threads of the epilogue.
__device__ __forceinline__ void stage_scales(float* to, const float* x_scale, int cols, int tn, int t) {
  for (int i = t; i < tn; i += kEpilogueThreads) to[i] = i < cols ? x_scale[i] : 0.f;
}
// The epilogue's threads meet; true if all of them are `ok`, so that after a wait that ran out none goes on without the
// others.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  int all;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n selp.s32 %0, 1, 0, q;\n}"
               : "=r"(all)
               : "r"((int)ok), "n"(kEpilogueThreads)
               : "memory");
  return all != 0;
}

// This warp's turns of 16 columns of an accumulator, f(first column, sums); the next turn's sums are on
// their way from tensor memory while f works.
template <typename F>
__device__ __forceinline__ void each16(uint32_t acc, int turn, int cols, F f) {
  float v[2][16];
  int c0 = 16 * turn;
  if (c0 < cols) tmem_ld16(acc + c0, v[0]);
#pragma unroll 1
  for (; c0 < cols; c0 += 64) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int c = c0 + 32 * b;
      if (c >= cols) break;
      tmem_wait_ld16(v[b]);
      if (c + 32 < cols) tmem_ld16(acc + c + 32, v[b ^ 1]);
      int sum[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] = __float_as_int(v[b][i]);
      f(c, sum);
    }
  }
}

// The end of a split tile: all parts' sums lie in shared memory as [token][128 channels]. This part's tokens are
// part, part + split, ...; a warp takes every tenth of them (four at a time, for loads in flight), a lane
// four neighbouring channels.
template <int CG>
__device__ __forceinline__ void exchange(const GemmParams& p, const uint8_t* ring, const float* xs, int part, int half, int n0, int m0,
                                         int cols, int warp, int lane) {
  constexpr int kWarps = kGemmThreads / 32, kBatch = 4;
  const int ch = n0 + 4 * lane, real = min(4, p.a.N - ch);   // channels of this lane that exist
  float ws[4], bias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ws[e] = e < real ? p.a.w_scale[ch + e] : 0.f;
    bias[e] = p.a.bias && e < real ? p.a.bias[ch + e] : 0.f;
  }
  const bool whole = real == 4 && (p.a.ldy & 3) == 0;        // four channels in one store
  for (int c0 = part + p.split * warp; c0 < cols; c0 += p.split * kWarps * kBatch) {
    int sum[kBatch][4] = {};
#pragma unroll 2
    for (int c = 0; c < p.split; ++c) {
      const uint32_t src = cluster_addr(ring, c * CG + half) + 16 * lane;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int tok = c0 + i * p.split * kWarps;
        if (tok < cols) {
          const int4 v = ld_cluster_v4(src + tok * 512);
          sum[i][0] += v.x; sum[i][1] += v.y; sum[i][2] += v.z; sum[i][3] += v.w;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int tok = c0 + i * p.split * kWarps;
      if (tok >= cols) break;
      const float x = xs[tok];
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = scaled(sum[i][e], x, ws[e]);
        if (p.a.bias) v[e] = biased(v[e], bias[e]);
      }
      const int64_t at = (int64_t)(m0 + tok) * p.a.ldy + ch;
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < real) store_y(p.a.y, p.a.y_type, at + e, v[e]);
      } else if (p.a.y_type == WR_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.a.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.y) + at) =
            p.a.y_type == WR_BF16 ? make_uint2(Bf16Out::two(v[0], v[1]), Bf16Out::two(v[2], v[3]))
                                  : make_uint2(F16Out::two(v[0], v[1]), F16Out::two(v[2], v[3]));
      }
    }
  }
}

// ---- split form: part r of tile t takes K blocks [r kb / split, (r + 1) kb / split). A part is a CTA, or
// with PAIR two neighbouring CTAs of the cluster (256 channels a tile).
template <bool PAIR>
__global__ void __launch_bounds__(kGemmThreads, 2)
    gemm_i8_split_kernel(const GemmParams p, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ GemmBars bars;
  constexpr int CG = PAIR ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int size = CG * p.split, rank = blockIdx.x % size, tile = blockIdx.x / size;
  const int part = rank / CG, half = rank % CG, leader = rank - half;
  const uint16_t mask = (uint16_t)(3 << leader);
  const int rg = tile / p.mt, mt = tile - rg * p.mt;
  const int n0 = (rg * CG + half) * 128, m0 = mt * p.tn;
  const int k0 = part * p.kb / p.split, k1 = (part + 1) * p.kb / p.split;
  const int b_rows = p.tn / CG;                       // tokens that this CTA loads
  const uint32_t a_bytes = 128 * 128, stage_bytes = a_bytes + (uint32_t)b_rows * 128;
  volatile int* abort_flag = &bars.abort_flag;
  const int q = warp & 3, turn = warp >= 6, row = 32 * q + lane, ch = n0 + row;
  const int cols = min(p.tn, p.a.M - m0);   // tokens of this tile
  float ws = 0.f, bias = 0.f;
  __shared__ float xs[256];

  // A CTA of its own fills the ring before it meets the other warps; a pair's copies complete on the
  // leader's barriers, which have to be there first.
  int k_next = k0;
  Ring last;   // of the loading thread
  grid_launch_dependents();
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&wmap);
      prefetch_tensormap(&xmap);
    }
    init_bars(bars, p.stages, 1);
    grid_dependency_wait();
    if (!PAIR && lane == 0) {
      for (int i = 0; i < p.stages && k_next < k1; ++i, ++k_next) {
        mbar_arrive_expect_tx(&bars.full[i], stage_bytes);
        tma_load_2d(ring + i * stage_bytes, &wmap, k_next * 128, n0, &bars.full[i]);
        tma_load_2d(ring + i * stage_bytes + a_bytes, &xmap, k_next * 128, m0, &bars.full[i]);
      }
    }
  } else if (warp == 1) {
    if (PAIR) tmem_alloc_pair(&bars.tmem_base, p.tmem_cols);
    else tmem_alloc(&bars.tmem_base, p.tmem_cols);
    grid_dependency_wait();
  } else {
    grid_dependency_wait();
    stage_scales(xs, p.a.x_scale + m0, cols, p.tn, threadIdx.x - 64);
    if (ch < p.a.N) {
      ws = p.a.w_scale[ch];
      if (p.a.bias) bias = p.a.bias[ch];
    }
  }
  fence_before_sync();
  if (PAIR) cluster_sync();
  else __syncthreads();
  fence_after_sync();
  const uint32_t tmem = bars.tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      Ring r;
      bool ok = true;
      for (int k = k0; k < k1; ++k, r.next(p.stages)) {
        if (k < k_next) continue;
        if (!(ok = mbar_wait_bg(&bars.empty[r.s], r.ph ^ 1, abort_flag, p.err, 501, p.wait_ns))) break;
        uint8_t* st = ring + r.s * stage_bytes;
        if (PAIR) {
          // both CTAs' copies complete on the leader's barrier
          if (half == 0) mbar_arrive_expect_tx(&bars.full[r.s], 2 * stage_bytes);
          const uint32_t bar = cluster_addr(&bars.full[r.s], leader);
          tma_load_2d_pair(st, &wmap, k * 128, n0, bar);
          tma_load_2d_pair(st + a_bytes, &xmap, k * 128, m0 + half * b_rows, bar);
        } else {
          mbar_arrive_expect_tx(&bars.full[r.s], stage_bytes);
          tma_load_2d(st, &wmap, k * 128, n0, &bars.full[r.s]);
          tma_load_2d(st + a_bytes, &xmap, k * 128, m0, &bars.full[r.s]);
        }
      }
      bars.copies = r.count;
      last = ok ? r : Ring{};
    }
  } else if (warp == 1) {
    if (half == 0) {   // a pair's leader issues for both CTAs
      const uint32_t idesc = idesc_i8s(128 * CG, p.tn);
      Ring r;
      bool ok = true;
      for (int k = k0; k < k1; ++k, r.next(p.stages)) {
        if (!(ok = warp_wait(&bars.full[r.s], r.ph, bars, p, 503))) break;
        fence_after_sync();
        const uint8_t* st = ring + r.s * stage_bytes;
        mma4_i8_ss_commit_elect<PAIR>(tmem, smem_desc_sw128(st), smem_desc_sw128(st + a_bytes), idesc, k != k0, &bars.empty[r.s], mask);
      }
      if (ok) {
        if (PAIR) mma_commit_pair_elect(&bars.acc_full[0], mask);
        else mma_commit_elect(&bars.acc_full[0]);
      }
      if (lane == 0) {
        bars.mmas = r.count;
        bars.accs = ok;
      }
    }
  } else {
    if (warp_wait(&bars.acc_full[0], 0, bars, p, 504)) {
      fence_after_sync();
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
      int* mine = reinterpret_cast<int*>(ring) + row;   // [token][channel]; every copy has been consumed
      if (p.split == 1) {
        each16(acc, turn, cols, [&](int c0, const int (&sum)[16]) {
          finish16(p.a, sum, xs + c0, m0 + c0, cols - c0, ch, lane, ws, bias);
        });
      } else {
        each16(acc, turn, cols, [&](int c0, const int (&sum)[16]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[(c0 + i) * 128] = sum[i];
        });
      }
    }
    fence_before_sync();
  }
  if (size > 1) pass_on_abort(bars, size, lane);
  if (p.split > 1) {
    cluster_sync();   // all parts are in shared memory
    if (!*abort_flag) exchange<CG>(p, ring, xs, part, half, n0, m0, cols, warp, lane);
  }
  if (threadIdx.x == 0 && last.count > 0 && !*abort_flag) {   // (here it has arrived; too late to raise the flag)
    uint32_t parity;
    uint64_t* bar = last_empty(bars, last, p.stages, parity);
    mbar_wait_drain(bar, parity);
  }
  fence_before_sync();
  if (size > 1) cluster_sync();   // nobody leaves while its shared memory (or tensor memory) is in use
  else __syncthreads();
  fence_after_sync();
  if (*abort_flag) {
    settle<PAIR>(&bars, p.stages, leader, stage_bytes, stage_bytes, 0);
    if (size > 1) cluster_sync();
    else __syncthreads();
  }
  if (warp == 1) {
    if (PAIR) tmem_dealloc_pair(tmem, p.tmem_cols);
    else tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ---- persistent form. Pairs take tiles in turn. With CUT whole rounds only, and each of the tiles that are left over
// (fewer than pairs) is cut into `cut` pieces of cut_tn tokens for as many pairs: 256 tokens of 19456 x 2560 are 76
// tiles for 74 pairs, 18.9 us in two rounds and 15.5 with pieces of 32 tokens (512 tokens 24.3 and 21.2).
struct Unit {
  int rg, m0, tn, cols;   // row group, first token, tokens of the MMA, real ones (0 or fewer: nothing to do)
};
template <bool CUT>
__device__ __forceinline__ Unit unit_of(const GemmParams& p, int u) {
  int t = u, from = 0, tn = p.tn;
  if (CUT && u >= p.whole) {
    const int v = u - p.whole;
    t = p.whole + v / p.cut;
    from = (v % p.cut) * p.cut_tn;
    tn = p.cut_tn;
  }
  Unit o;
  o.rg = t / p.mt;
  o.m0 = (t - o.rg * p.mt) * p.tn + from;
  o.tn = tn;
  o.cols = min(CUT ? min(tn, p.tn - from) : tn, p.a.M - o.m0);
  return o;
}

template <bool CUT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_i8_persistent_kernel(const GemmParams p, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                              const __grid_constant__ CUtensorMap xmap_cut) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ GemmBars bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int worker = blockIdx.x / 2, G = gridDim.x / 2;
  const uint32_t a_bytes = 128 * 128, stage_bytes = a_bytes + (uint32_t)p.tn / 2 * 128;   // each CTA loads half of the tokens
  volatile int* abort_flag = &bars.abort_flag;
  __shared__ float xs[2][256];
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&wmap);
      prefetch_tensormap(&xmap);
      if (CUT) prefetch_tensormap(&xmap_cut);
    }
    init_bars(bars, p.stages, 2 * kEpilogueThreads / 32);
  }
  grid_launch_dependents();
  if (warp == 1) tmem_alloc_pair(&bars.tmem_base, p.tmem_cols);
  fence_before_sync();
  grid_dependency_wait();
  cluster_sync();
  fence_after_sync();
  const uint32_t tmem = bars.tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      Ring r;
      bool ok = true;
      for (int u = worker; ok && u < p.units; u += G) {
        const Unit o = unit_of<CUT>(p, u);
        if (CUT && o.cols <= 0) continue;
        const int n0 = (o.rg * 2 + (int)rank) * 128, m0 = o.m0 + (int)rank * (o.tn / 2);
        const CUtensorMap* xm = CUT && u >= p.whole ? &xmap_cut : &xmap;
        const uint32_t bytes = a_bytes + (uint32_t)o.tn / 2 * 128;
        for (int k = 0; k < p.kb; ++k, r.next(p.stages)) {
          if (!(ok = mbar_wait_bg(&bars.empty[r.s], r.ph ^ 1, abort_flag, p.err, 511, p.wait_ns))) break;
          uint8_t* st = ring + r.s * stage_bytes;
          // both CTAs' copies complete on the leader's barrier
          if (rank == 0) mbar_arrive_expect_tx(&bars.full[r.s], 2 * bytes);
          const uint32_t bar = cluster_addr(&bars.full[r.s], 0);
          tma_load_2d_pair(st, &wmap, k * 128, n0, bar);
          tma_load_2d_pair(st + a_bytes, xm, k * 128, m0, bar);
        }
      }
      bars.copies = r.count;
      if (ok) {
        uint32_t parity;
        uint64_t* bar = last_empty(bars, r, p.stages, parity);
        mbar_wait_bg(bar, parity, abort_flag, p.err, 515, p.wait_ns);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {   // the leader issues for both CTAs
      Ring r;
      uint32_t n = 0;   // accumulators committed
      bool ok = true;
      for (int u = worker; ok && u < p.units; u += G) {
        const Unit o = unit_of<CUT>(p, u);
        if (CUT && o.cols <= 0) continue;
        const uint32_t d = n & 1, idesc = idesc_i8s(256, o.tn);
        if (!(ok = warp_wait(&bars.acc_empty[d], ((n >> 1) & 1) ^ 1, bars, p, 512))) break;
        fence_after_sync();
        for (int k = 0; k < p.kb; ++k, r.next(p.stages)) {
          if (!(ok = warp_wait(&bars.full[r.s], r.ph, bars, p, 513))) break;
          fence_after_sync();
          const uint8_t* st = ring + r.s * stage_bytes;
          mma4_i8_ss_commit_elect<true>(tmem + d * p.tn, smem_desc_sw128(st), smem_desc_sw128(st + a_bytes), idesc, k != 0,
                                        &bars.empty[r.s], 3);
        }
        if (!ok) break;
        mma_commit_pair_elect(&bars.acc_full[d], 3);
        ++n;
      }
      if (lane == 0) {
        bars.mmas = r.count;
        bars.accs = n;
      }
    }
  } else {
    // The scales of a tile are read while the one before it is written (8 rounds of 256 x 32 tokens and one block of
    // K: 9.8 us, read at a tile's start 10.4).
    const int q = warp & 3, turn = (warp - 2) >> 2, te = threadIdx.x - 64;
    float ws_next, bias_next, xs_next;
    auto scales = [&](const Unit& o) {
      const int ch = (o.rg * 2 + (int)rank) * 128 + 32 * q + lane;
      ws_next = ch < p.a.N ? p.a.w_scale[ch] : 0.f;
      bias_next = p.a.bias && ch < p.a.N ? p.a.bias[ch] : 0.f;
      xs_next = te < o.cols ? p.a.x_scale[o.m0 + te] : 0.f;
    };
    uint32_t n = 0;
    int u = worker;
    Unit o = unit_of<CUT>(p, u);
    scales(o);
    for (; u < p.units; u += G) {
      const Unit now = o;
      const float ws = ws_next, bias = bias_next;
      const uint32_t d = n & 1;
      if (te < 256) xs[d][te] = xs_next;
      if (u + G < p.units) scales(o = unit_of<CUT>(p, u + G));
      if (CUT && now.cols <= 0) continue;
      const int ch = (now.rg * 2 + (int)rank) * 128 + 32 * q + lane, m0 = now.m0, cols = now.cols;
      // (xs[d] was last read two tiles ago, before the other one's barrier)
      if (!epilogue_all(warp_wait(&bars.acc_full[d], (n >> 1) & 1, bars, p, 514))) break;
      fence_after_sync();
      const uint32_t acc = tmem + d * p.tn + ((uint32_t)(32 * q) << 16);
      each16(acc, turn, cols, [&](int c0, const int (&sum)[16]) {
        finish16(p.a, sum, xs[d] + c0, m0 + c0, cols - c0, ch, lane, ws, bias);
      });
      fence_before_sync();
      __syncwarp();
      // Relaxed: only the reads of tensor memory come before it, and they are done. A release would wait until y is
      // written (12.2 us become 17.3, 8 rounds of 256 x 32 tokens and four blocks of K).
      if (lane == 0) mbar_arrive_cluster_relaxed(cluster_addr(&bars.acc_empty[d], 0));
      ++n;
    }
  }
  pass_on_abort(bars, 2, lane);
  fence_before_sync();
  cluster_sync();
  fence_after_sync();
  if (*abort_flag) {
    const uint32_t rounds = worker < p.whole ? (p.whole - 1 - worker) / G + 1 : 0;   // whole tiles of this pair
    settle<true>(&bars, p.stages, 0, stage_bytes, a_bytes + (uint32_t)p.cut_tn / 2 * 128, rounds * p.kb);
    cluster_sync();
  }
  if (warp == 1) tmem_dealloc_pair(tmem, p.tmem_cols);
}

constexpr int kSMs = 148;

// Shared memory of a CTA. A CTA that finds too little tensor memory waits until another one leaves; the CTAs of
// a cluster wait for one another. Two clusters (calls on two streams) that held tensor memory on one SM each
// and waited for it on the other's would wait for good. So a CTA of a cluster claims its SM's shared memory
// whole and never meets another of these CTAs there; one on its own claims as large a share as of the
// tensor memory (222 KB for 512 columns), so that whatever fits the SM finds its columns. The ring takes what
// the claim allows.
constexpr int kClaimPerColumn = 222 * 1024 / 512;
constexpr int kRing = 256 * kClaimPerColumn - 1024, kDeepRing = 512 * kClaimPerColumn - 1024;   // (1024: alignment)

// Clusters of 1 .. 8 CTAs that run at once with one CTA an SM (a cluster stays inside a GPC, so sizes that do
// not divide its SMs leave some idle; cudaOccupancyMaxActiveClusters on this part).
constexpr int kClusters[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};

// Shared memory limits are set once per device and kernel.
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = own_error(cudaGetDevice(&dev));
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = own_error(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  return cudaSuccess;
}

// Tokens of a piece when the tiles of tn tokens that are left over are cut: each CTA of a pair loads half of them.
constexpr int cut_tokens(int tn, int cut) { return ((tn + cut - 1) / cut + 31) / 32 * 32; }

// Expected time of a plan in microseconds, in a stream of such calls. The form follows the machine (bytes into
// an SM, clocks of the tensor core, memory, a start and an end for each tile); the constants are fitted to the
// times of all plans on 416 shapes (M 8 .. 4096, N 64 .. 19456, K 64 .. 16384). On 147 other shapes the plan
// it picked took 2 % longer than the best one in the geometric mean; one CTA a tile with the fewest token tiles
// and K whole takes 55 % longer.
double expected_us(const GemmI8Plan& p, int64_t M, int64_t N, int64_t K) {
  const int cg = 1 + p.pair, tn = p.tn;
  // weights that several token tiles read come from memory more than once now and then
  const double memory = ((p.mt > 1 ? 1.23 : 1.0) * N * K + M * K + 2.0 * M * N) / 5.5e6;
  auto tensor = [](int t) { return 2.0 * t / 1900; };              // one block: 8192 products a clock
  if (p.persistent) {
    auto round = [&](int t) { return std::max(p.kb * std::max(tensor(t), (16384 + 64.0 * t) / 96.6e3), 0.19 + 0.0153 * t); };
    const int64_t rounds = p.tiles / (kSMs / 2), left = p.tiles % (kSMs / 2);
    const double last = left == 0 ? 0 : round(p.cut > 1 ? cut_tokens(tn, p.cut) : tn);
    return 3.0 + std::max(rounds * round(tn) + last, memory) + 0.009 * tn;
  }
  // two CTAs on their own share an SM; clusters run at once
  const bool alone = p.tiles <= kClusters[cg * p.split];
  const int64_t waves = alone ? 1 : (p.tiles + 2 * kSMs - 1) / (2 * kSMs), even = (p.tiles + kSMs - 1) / kSMs;
  const int64_t most = alone ? 1 : std::max(2 * waves - 1, std::min(2 * waves, even));   // CTAs of the busiest SM
  const int blocks = (p.kb + p.split - 1) / p.split;
  const double block = std::max(tensor(tn), (16384 + 128.0 * tn / cg) / 123e3);
  double t = 0.54 + 0.62 * p.pair + std::max(most * blocks * block, memory) + waves * 1.85;
  t += p.split > 1 ? 0.59 + 0.015 * cg * cg * p.split * p.split + waves * 0.025 * tn : waves * 0.021 * tn;
  return t;
}

}  // namespace

bool plan_gemm_i8(int64_t M, int64_t N, int64_t K, GemmI8Plan* p) {
  GemmI8Plan o{};
  o.kb = (int)((K + 127) / 128);
  o.cut = 1;
  double best = 0;
  bool any = false;
  auto offer = [&] {
    const double t = expected_us(o, M, N, K);
    if (any && t >= best) return;
    any = true;
    best = t;
    *p = o;
  };
  const int64_t mt0 = (M + 255) / 256, mt1 = std::min<int64_t>((M + 15) / 16, mt0 + 7);
  for (int64_t mt = mt0; mt <= mt1; ++mt) {
    for (o.pair = 0; o.pair < (N > 128 ? 2 : 1); ++o.pair) {
      const int cg = 1 + o.pair, step = 16 * cg;
      o.tn = (int)(((M + mt - 1) / mt + step - 1) / step * step);
      o.mt = (int)((M + o.tn - 1) / o.tn);
      const int64_t tiles = o.mt * ((N + 128 * cg - 1) / (128 * cg));
      if (tiles > (1 << 26)) return false;
      o.tiles = (int)tiles;
      o.persistent = 0;
      for (o.split = 1; o.split <= std::min(8 / cg, o.kb); ++o.split)
        if (cg * o.split == 1 || o.tiles <= kClusters[cg * o.split]) offer();
      o.split = 1;
      if (o.pair) {
        o.persistent = 1;
        offer();
        // what is left after whole rounds, cut for more pairs
        const int left = o.tiles % (kSMs / 2);
        if (o.tiles > kSMs / 2 && left)
          for (o.cut = std::min(o.tn / 32, kSMs / 2 / left); o.cut > 1; --o.cut) offer();
        o.cut = 1;
      }
    }
  }
  return true;
}

cudaError_t launch_gemm_i8(const GemmI8Args& a, const GemmI8Plan& pl, int* err, cudaStream_t stream, uint64_t wait_ns) {
  const int cg = 1 + pl.pair;
  GemmParams p{};
  p.a = a;
  p.tn = pl.tn;
  p.mt = pl.mt;
  p.kb = pl.kb;
  p.split = pl.split;
  p.cut = pl.cut;
  p.cut_tn = cut_tokens(pl.tn, pl.cut);
  p.whole = pl.cut > 1 ? pl.tiles - pl.tiles % (kSMs / 2) : pl.tiles;
  p.units = p.whole + (pl.tiles - p.whole) * pl.cut;
  const int stage = 128 * 128 + pl.tn / cg * 128;
  const int cluster = pl.persistent ? 2 : cg * pl.split;
  const int64_t ctas = (int64_t)(pl.persistent ? std::min(p.units, kSMs / 2) : pl.tiles) * cluster;
  // CTAs that have an SM for themselves take the deeper ring
  const int room = cluster > 1 || pl.tiles <= kClusters[1] ? kDeepRing : kRing;
  p.stages = std::min({kMaxStages, room / stage, std::max(1, (pl.kb + pl.split - 1) / pl.split * (pl.persistent ? kMaxStages : 1))});
  p.tmem_cols = 32;
  while (p.tmem_cols < (pl.persistent ? 2 : 1) * pl.tn) p.tmem_cols *= 2;   // two accumulators in the persistent form
  p.err = err;
  p.wait_ns = wait_ns;
  CUtensorMap wmap, xmap, xmap_cut;
  if (!encode_bytes_2d(&wmap, a.w, a.K, a.N, a.ldw, 128) || !encode_bytes_2d(&xmap, a.x, a.K, a.M, a.ldx, pl.tn / cg) ||
      (pl.cut > 1 && !encode_bytes_2d(&xmap_cut, a.x, a.K, a.M, a.ldx, p.cut_tn / 2)))
    return cudaErrorInvalidValue;
  static std::atomic<bool> done[4][64];
  // the ring, or the sums that replace it at the end of a split tile
  const int ring = std::max(p.stages * stage, pl.split > 1 ? pl.tn * 512 : 0);
  const int smem = std::max(ring + 1024, (cluster > 1 ? 512 : p.tmem_cols) * kClaimPerColumn);
  auto run = [&](auto kern, int form, auto... maps) {
    const cudaError_t e = allow_smem(kern, kDeepRing + 1024, done[form]);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, dim3((unsigned)ctas), dim3(kGemmThreads), (size_t)smem, cluster, stream, p, maps...);
  };
  if (pl.cut > 1) return run(gemm_i8_persistent_kernel<true>, 3, wmap, xmap, xmap_cut);
  if (pl.persistent) return run(gemm_i8_persistent_kernel<false>, 2, wmap, xmap, xmap);
  return pl.pair ? run(gemm_i8_split_kernel<true>, 1, wmap, xmap) : run(gemm_i8_split_kernel<false>, 0, wmap, xmap);
}

cudaError_t launch_gemv_i8(const GemmI8Args& a, cudaStream_t stream) {
  return a.M == 1 ? run_gemv<1>(a, stream) : run_gemv<2>(a, stream);
}

cudaError_t launch_few_i8(const GemmI8Args& a, cudaStream_t stream) {
  // Four turns at once and two CTAs an SM, or two turns and a third CTA, by what lets all rows run at once (8
  // tokens: 4096 x 2560 3.3 and 3.9 us, 4096 x 9728 8.8 and 10.5; 6144 x 2560 5.6 and 4.0). With few of rows
  // and bytes, and for 2 KB behind 7104 rows, two turns are enough (1024 x 2048: 2.6 and 2.2; 8192 x 2048: 5.6
  // and 4.9, of 4096 bytes 8.1 and 9.2).
  const bool deep = a.N <= kFewAtOnce / 3 * 2 ? a.K > 2048 || a.N > 2048 : a.N > kFewAtOnce && a.K > 2048;
  const auto kern = a.M > 8 ? few_i8_kernel<2, 2, 2> : deep ? few_i8_kernel<4, 2, 1> : few_i8_kernel<2, 3, 1>;
  return launch_overlapped(kern, dim3((unsigned)((a.N + 15) / 16)), dim3(kFewThreads), 0, 1, stream, a);
}

}  // namespace wr
