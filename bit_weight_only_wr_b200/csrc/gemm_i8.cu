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
#include "tc_common.cuh"
#include "tc_kernels.cuh"

namespace wr {
namespace {

using namespace tc;

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

// ---------------------------------------------------------------- more tokens: tcgen05 kind::i8

// The channels are the rows of the MMA (A, 128 a CTA), the tokens its columns (B), so that a thread of the
// epilogue owns one channel and a warp writes 32 neighbouring ones. A tile is 128 channels (256 for a
// CTA pair) by tn tokens; its K is cut in blocks of 128 bytes, one stage of the ring each (TMA, 128-byte
// swizzle, zeros behind the ends of K, M and N).
// Work: worker c (a CTA or a pair) first takes blocks [c S / G, (c + 1) S / G) of the first sk_tiles
// tiles (S blocks in all), then whole tiles sk_tiles + c, + G, ... A tile cut by a range's end is
// finished by whichever of its workers comes last: each adds its int32 sums to the tile's in the
// workspace (zero between calls), and the last reads them. The sums are exact, so the order of the
// additions changes nothing.
// Warps: 0 loads (TMA), 1 issues the MMAs, 2-5 are the epilogue (TMEM lanes 32 (warp % 4) ..).
constexpr int kGemmThreads = 192;
constexpr int kMaxStages = 10;
constexpr int kSmemRing = 208 * 1024;

struct GemmBars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};

struct GemmParams {
  GemmI8Args a;
  int tn, mt, kb, tiles, sk_tiles, stages, tmem_cols;
  int* counter;      // one per epilogue warp of each worker's CTAs, zero between calls
  int* partial;      // [worker][CTA of the pair][tn][128]: sums of the cut tile that starts in its range, zero between calls
  int* err;
};

struct Piece {
  int tile, k0, k1;
};
// The pieces of worker c in order.
struct Pieces {
  int u, u1, kb, next, tiles, G;
  __device__ __forceinline__ Pieces(const GemmParams& p, int c, int G_) : kb(p.kb), tiles(p.tiles), G(G_) {
    const int S = p.sk_tiles * p.kb;
    u = (int)((int64_t)c * S / G);
    u1 = (int)((int64_t)(c + 1) * S / G);
    next = p.sk_tiles + c;
  }
  __device__ __forceinline__ bool get(Piece& o) {
    if (u < u1) {
      o.tile = u / kb;
      o.k0 = u - o.tile * kb;
      o.k1 = min(kb, o.k0 + (u1 - u));
      u += o.k1 - o.k0;
      return true;
    }
    if (next >= tiles) return false;
    o.tile = next;
    o.k0 = 0;
    o.k1 = kb;
    next += G;
    return true;
  }
};

// x_scale of 16 tokens (`left` of them real; the address is 64-byte aligned).
__device__ __forceinline__ void load_scales16(const float* xs, int left, float v[16]) {
  if (left >= 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(xs) + i);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < left ? __ldg(xs + i) : 0.f;
  }
}

// Writes this thread's channel of 16 tokens from token m on (`left` of them real): v plus the bias. A
// warp holds 32 neighbouring channels, so a token's store is 128 contiguous bytes of fp32. For a
// 16-bit y neighbouring lanes exchange halves, so that even lanes store pairs of channels of the even
// tokens and odd lanes those of the odd ones (half the stores; needs rows that start on 4 bytes).
__device__ __forceinline__ void store16(const GemmI8Args& a, int m, int left, int ch, int lane, float v[16], float bias) {
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += bias;
  }
  if (a.y_type == WR_F32) {
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
    return;
  }
  uint32_t h[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    h[i] = a.y_type == WR_BF16 ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v[i]))
                               : (uint32_t)__half_as_ushort(__float2half_rn(v[i]));
  uint16_t* y = static_cast<uint16_t*>(a.y) + (int64_t)m * a.ldy + ch;
  const bool odd = lane & 1;
  if ((a.ldy & 1) == 0 && (ch - lane) + 32 <= a.N && left >= 16) {
    // the warp's 32 channels are all real: lane pairs cover them
    uint32_t* y2 = reinterpret_cast<uint32_t*>(y - odd) + (odd ? a.ldy / 2 : 0);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? h[i] : h[i + 1], 1);
      y2[(i / 2) * a.ldy] = odd ? (got | h[i + 1] << 16) : (h[i] | got << 16);
    }
    return;
  }
  if (ch >= a.N) return;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < left) y[i * a.ldy] = (uint16_t)h[i];
}

template <bool PAIR>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_i8_kernel(const GemmParams p, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ GemmBars bars;
  constexpr int CG = PAIR ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const int worker = blockIdx.x / CG, G = gridDim.x / CG;
  const int b_rows = p.tn / CG;                       // tokens that this CTA loads
  const uint32_t a_bytes = 128 * 128, b_bytes = (uint32_t)b_rows * 128, stage_bytes = a_bytes + b_bytes;
  volatile int* abort_flag = &bars.abort_flag;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 4 * CG);
    }
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (PAIR) tmem_alloc_pair(&bars.tmem_base, p.tmem_cols);
    else tmem_alloc(&bars.tmem_base, p.tmem_cols);
  }
  fence_before_sync();
  if (PAIR) cluster_sync();
  else __syncthreads();
  fence_after_sync();
  const uint32_t tmem = bars.tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tensormap(&wmap);
      prefetch_tensormap(&xmap);
      uint32_t it = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      Pieces pieces(p, worker, G);
      for (Piece w; ok && pieces.get(w);) {
        const int rg = w.tile / p.mt, mt = w.tile - rg * p.mt;
        const int n0 = (rg * CG + (int)rank) * 128, m0 = mt * p.tn + (int)rank * b_rows;
        for (int k = w.k0; k < w.k1; ++k) {
          if (!(ok = mbar_wait_bg(&bars.empty[s], ph ^ 1, abort_flag, p.err, 501))) break;
          uint8_t* a_st = ring + s * stage_bytes;
          if (PAIR) {
            // both CTAs' copies complete on the leader's barrier
            if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], 2 * stage_bytes);
            const uint32_t bar = cluster_addr(&bars.full[s], 0);
            tma_load_2d_pair(a_st, &wmap, k * 128, n0, bar);
            tma_load_2d_pair(a_st + a_bytes, &xmap, k * 128, m0, bar);
          } else {
            mbar_arrive_expect_tx(&bars.full[s], stage_bytes);
            tma_load_2d(a_st, &wmap, k * 128, n0, &bars.full[s]);
            tma_load_2d(a_st + a_bytes, &xmap, k * 128, m0, &bars.full[s]);
          }
          ++it;
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok && rank == 0) {   // let the copies in flight land before the CTA leaves
        const uint32_t n = it < (uint32_t)p.stages ? it : (uint32_t)p.stages;
        for (uint32_t i = 0; i < n; ++i) {
          const uint32_t j = it - 1 - i;
          if (!mbar_wait_drain(&bars.full[j % p.stages], (j / p.stages) & 1)) break;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the pair's leader)
    if (rank == 0) {
      const uint32_t idesc = idesc_i8s(128 * CG, p.tn);
      int s = 0;
      uint32_t ph = 0, n = 0;
      bool ok = true;
      Pieces pieces(p, worker, G);
      for (Piece w; ok && pieces.get(w); ++n) {
        const uint32_t d = n & 1;
        if (!(ok = mbar_wait_bg(&bars.acc_empty[d], ((n >> 1) & 1) ^ 1, abort_flag, p.err, 502))) break;
        for (int k = w.k0; k < w.k1; ++k) {
          if (!(ok = mbar_wait_bg(&bars.full[s], ph, abort_flag, p.err, 503))) break;
          fence_after_sync();
          const uint8_t* a_st = ring + s * stage_bytes;
          mma4_i8_ss_commit_elect<PAIR>(tmem + d * p.tn, smem_desc_sw128(a_st), smem_desc_sw128(a_st + a_bytes), idesc, k != w.k0,
                                        &bars.empty[s]);
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (PAIR) mma_commit_pair_elect(&bars.acc_full[d]);
        else mma_commit_elect(&bars.acc_full[d]);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int S = p.sk_tiles * p.kb;
    uint32_t n = 0;
    Pieces pieces(p, worker, G);
    for (Piece w; pieces.get(w); ++n) {
      const uint32_t d = n & 1;
      const int rg = w.tile / p.mt, mt = w.tile - rg * p.mt;
      const int ch = (rg * CG + (int)rank) * 128 + 32 * q + lane, m0 = mt * p.tn;
      const int cols = min(p.tn, p.a.M - m0);         // tokens of this tile
      const float ws = ch < p.a.N ? __ldg(p.a.w_scale + ch) : 0.f;
      const float bias = p.a.bias && ch < p.a.N ? __ldg(p.a.bias + ch) : 0.f;
      if (!mbar_wait(&bars.acc_full[d], (n >> 1) & 1, abort_flag, p.err, 504)) break;
      fence_after_sync();
      const uint32_t acc = tmem + d * p.tn + ((uint32_t)(32 * q) << 16);
      auto release = [&]() {   // the accumulator may be overwritten
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(cluster_addr(&bars.acc_empty[d], 0));
          else mbar_arrive(&bars.acc_empty[d]);
        }
      };
      if (w.k0 == 0 && w.k1 == p.kb) {
        for (int c0 = 0; c0 < cols; c0 += 16) {
          float v[16];
          tmem_ld16(acc + c0, v);
          float xs[16];
          load_scales16(p.a.x_scale + m0 + c0, cols - c0, xs);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = (float)__float_as_int(v[i]) * xs[i] * ws;
          store16(p.a, m0 + c0, cols - c0, ch, lane, v, bias);
        }
        release();
        continue;
      }
      // a piece of a tile: add it to the tile's sums in the workspace; the last piece to arrive writes y
      const int tb = w.tile * p.kb;
      const int c_first = (int)((((int64_t)tb + 1) * G - 1) / S), c_last = (int)(((int64_t)(tb + p.kb) * G - 1) / S);
      int* sums = p.partial + ((int64_t)c_first * CG + rank) * p.tn * 128 + 32 * q + lane;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        tmem_ld16(acc + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) atomicAdd(sums + (c0 + i) * 128, __float_as_int(v[i]));
      }
      release();
      __threadfence();
      __syncwarp();
      int* counter = p.counter + (c_first * CG + (int)rank) * 4 + q;
      int seen = 0;
      if (lane == 0) seen = atomicAdd(counter, 1);
      seen = __shfl_sync(0xffffffffu, seen, 0);
      if (seen != c_last - c_first) continue;
      __threadfence();
      if (lane == 0) *counter = 0;
      for (int c0 = 0; c0 < cols; c0 += 32) {
        int t[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) t[i] = c0 + i < p.tn ? __ldcg(sums + (c0 + i) * 128) : 0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c0 + i < p.tn) __stcg(sums + (c0 + i) * 128, 0);
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          if (c0 + h >= cols) break;
          float v[16], xs[16];
          load_scales16(p.a.x_scale + m0 + c0 + h, cols - c0 - h, xs);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = (float)t[h + i] * xs[i] * ws;
          store16(p.a, m0 + c0 + h, cols - c0 - h, ch, lane, v, bias);
        }
      }
    }
  }
  fence_before_sync();
  if (PAIR) cluster_sync();
  else __syncthreads();
  fence_after_sync();
  if (warp == 1) {
    if (PAIR) tmem_dealloc_pair(tmem, p.tmem_cols);
    else tmem_dealloc(tmem, p.tmem_cols);
  }
}

constexpr int kGemmSmem = kSmemRing + 1024;
constexpr int kSMs = 148;

template <bool PAIR>
cudaError_t run_gemm(const GemmParams& p, int workers, const CUtensorMap& wmap, const CUtensorMap& xmap, cudaStream_t stream) {
  // per device: an attribute set on one does not hold on another
  const cudaError_t e = cudaFuncSetAttribute(gemm_i8_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(workers * (PAIR ? 2 : 1)));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  if (PAIR) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, gemm_i8_kernel<PAIR>, p, wmap, xmap);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

bool plan_gemm_i8(int64_t M, int64_t N, int64_t K, GemmI8Plan* p) {
  *p = GemmI8Plan{};
  p->pair = 0;
  const int cg = 1, step = 16;
  const int64_t mt = (M + 255) / 256;
  p->tn = (int)(((M + mt - 1) / mt + step - 1) / step * step);
  const int64_t tiles = mt * ((N + 128 * cg - 1) / (128 * cg));
  if (tiles > (1 << 30)) return false;
  p->mt = (int)mt;
  p->tiles = (int)tiles;
  p->kb = (int)((K + 127) / 128);
  const int slots = kSMs / cg;
  p->workers = (int)std::min<int64_t>(slots, tiles * p->kb);
  const int64_t waves = tiles / p->workers, rest = tiles % p->workers;
  if (rest != 0) p->sk_tiles = (int)(rest + (waves > 0 ? p->workers : 0));
  if (p->sk_tiles > 0) {
    p->counter_bytes = align256((size_t)p->workers * cg * 4 * sizeof(int));
    p->workspace_bytes = p->counter_bytes + (size_t)p->workers * cg * p->tn * 128 * sizeof(int);
  }
  return true;
}

cudaError_t launch_gemm_i8(const GemmI8Args& a, const GemmI8Plan& pl, void* workspace, int* err, cudaStream_t stream) {
  const int cg = pl.pair ? 2 : 1;
  GemmParams p{};
  p.a = a;
  p.tn = pl.tn;
  p.mt = pl.mt;
  p.kb = pl.kb;
  p.tiles = pl.tiles;
  p.sk_tiles = pl.sk_tiles;
  p.stages = std::min(kMaxStages, kSmemRing / (128 * 128 + pl.tn / cg * 128));
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * pl.tn) p.tmem_cols *= 2;
  p.counter = static_cast<int*>(workspace);
  p.partial = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + pl.counter_bytes);
  p.err = err;
  CUtensorMap wmap, xmap;
  if (!encode_bytes_2d(&wmap, a.w, a.K, a.N, a.ldw, 128) || !encode_bytes_2d(&xmap, a.x, a.K, a.M, a.ldx, pl.tn / cg))
    return cudaErrorInvalidValue;
  return pl.pair ? run_gemm<true>(p, pl.workers, wmap, xmap, stream) : run_gemm<false>(p, pl.workers, wmap, xmap, stream);
}

cudaError_t launch_gemv_i8(const GemmI8Args& a, cudaStream_t stream) {
  if (a.M == 1) return run_gemv<1, 1>(a, stream);
  if (a.M == 2) return run_gemv<2, 2>(a, stream);
  if (a.M <= 4) return run_gemv<4, 4>(a, stream);
  return run_gemv<4, 8>(a, stream);
}

}  // namespace wr
