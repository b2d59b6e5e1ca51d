// norm.cuh -- residual addition + root-mean-square norm whose output leaves as
// E4M3 codes, and its backward pass (sm_100a, HBM-bound).
//
//   h    = bf16(x + residual)                (h = x without a residual)
//   rstd = 1 / sqrt(mean_c h^2 + eps)        fp32
//   y    = (h * rstd) * gamma                fp32
//   codes and scales of y as the quantisers write them, but of the fp32 y:
//   the only rounding of y is the one to E4M3.
// Backward, with dy the gradient of y and dres the one that reaches h directly
// (the residual stream):
//   g = dy * gamma,  xh = h * rstd,  m = mean_c(g * xh)
//   dh = bf16(rstd * (g - xh * m) + dres),   dgamma_c = sum_rows dy * xh  (fp32)
//
// A row is held in registers by the threads that share it (8 columns = one
// 16-byte load per thread and chunk), so x and the residual are read once; the
// row sum is a warp shuffle plus, when several warps share a row, one step
// through shared memory. 16 consecutive threads hold one 1x128 group.
// Column-wise codes need all 128 rows' rstd first: norm_col_kernel makes a
// second pass over h in 128x128 tiles, last rows first, while h is still in L2.
#pragma once

#include "../common.cuh"
#include "tile_quant.cuh"

namespace fp8bw {
namespace layer {

// ---------------------------------------------------------------- helpers
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint4 ld16(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// Read once, not needed again: keep it from displacing what is re-read from L2.
__device__ __forceinline__ uint4 ld16_stream(const void* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}

// A second read that the compiler must not merge with the first (whose
// registers would then have to live until here).
__device__ __forceinline__ uint4 ld16_again(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  f[0] = bf16_lo(w.x);
  f[1] = bf16_hi(w.x);
  f[2] = bf16_lo(w.y);
  f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z);
  f[5] = bf16_hi(w.z);
  f[6] = bf16_lo(w.w);
  f[7] = bf16_hi(w.w);
}

// Eight consecutive norm weights (bf16 or fp32) starting at column c.
__device__ __forceinline__ void load_gamma8(const void* gamma, int is_f32, int64_t c,
                                            float (&g)[8]) {
  if (is_f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(gamma) + c);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
    g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
  } else {
    unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(gamma) + c)), g);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ---------------------------------------------------------------- forward, row-wise
struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;   // may be null: h = x
  const void* gamma;
  int gamma_f32;
  int64_t row0, row_end;      // this launch's rows of [0, rows_pad)
  int64_t rows, rows_pad, cols;
  float eps;
  uint16_t* h;                // written when there is a residual
  float* rstd;                // may be null
  uint16_t* y;                // bf16 output, may be null
  uint8_t* q;                 // row-wise codes, may be null
  float* s;                   // their scales [ceil(cols/128)][rows_pad]
  int tpr;                    // threads per row, a multiple of 32
};

constexpr int kNormMaxWarps = 32;

// V chunks of 8 columns per thread; blockDim = groups x tpr, one row each.
template <int V, bool POW2>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512)
    rmsnorm_row_kernel(const NormArgs a) {
  __shared__ float part[kNormMaxWarps];
  launch_dependents();
  grid_dependency_wait();
  const int tpr = a.tpr;
  const int grp = threadIdx.x / tpr;
  const int t = threadIdx.x - grp * tpr;
  const int groups = blockDim.x / tpr;
  const int64_t row = a.row0 + static_cast<int64_t>(blockIdx.x) * groups + grp;
  const bool live = row < a.rows && row < a.row_end;
  const int chunks = static_cast<int>(a.cols >> 3);
  const int64_t base = row * a.cols;

  uint4 h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + v * tpr;
    h[v] = make_uint4(0u, 0u, 0u, 0u);
    if (live && c < chunks) h[v] = ld16_stream(a.x + base + 8 * static_cast<int64_t>(c));
  }
  if (a.residual != nullptr) {
    uint4 r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * tpr;
      r[v] = make_uint4(0u, 0u, 0u, 0u);
      if (live && c < chunks) r[v] = ld16_stream(a.residual + base + 8 * static_cast<int64_t>(c));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * tpr;
      float f[8], e[8];
      unpack8(h[v], f);
      unpack8(r[v], e);
      h[v] = make_uint4(pack_bf16(f[0] + e[0], f[1] + e[1]), pack_bf16(f[2] + e[2], f[3] + e[3]),
                        pack_bf16(f[4] + e[4], f[5] + e[5]), pack_bf16(f[6] + e[6], f[7] + e[7]));
      if (live && c < chunks)
        *reinterpret_cast<uint4*>(a.h + base + 8 * static_cast<int64_t>(c)) = h[v];
    }
  }

  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f[8];
    unpack8(h[v], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
  }
  ss = warp_sum(ss);
  const int wpr = tpr >> 5;
  if (wpr > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < wpr; ++w) ss += part[grp * wpr + w];
  }
  const float rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(ss, static_cast<float>(a.cols)) + a.eps));
  if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
  if (a.q == nullptr && a.y == nullptr) return;

#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + v * tpr;
    const bool in = c < chunks;
    float y[8], g[8];
    unpack8(h[v], y);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 0.0f;
    if (live && in) load_gamma8(a.gamma, a.gamma_f32, 8 * static_cast<int64_t>(c), g);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = live && in ? (y[j] * rstd) * g[j] : 0.0f;
    if (a.y != nullptr && live && in)
      *reinterpret_cast<uint4*>(a.y + base + 8 * static_cast<int64_t>(c)) =
          make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                     pack_bf16(y[6], y[7]));
    if (a.q != nullptr) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      float qs, s;
      scale_of<POW2>(m, qs, s);
      if (in && row < a.row_end) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= qs;
        *reinterpret_cast<uint2*>(a.q + base + 8 * static_cast<int64_t>(c)) = encode8(y);
        if ((c & 15) == 0) a.s[static_cast<int64_t>(c >> 4) * a.rows_pad + row] = s;
      }
    }
  }
}

// ---------------------------------------------------------------- forward, column-wise
// y of a 128x128 tile of h, from the rows' rstd, to column-wise codes.
struct NormColArgs {
  const float* rstd;
  const void* gamma;
  int gamma_f32;
  int64_t rows, rows_pad, cols;
  int tr0;                    // first row tile of this launch
  int tiles_r, tiles_c;
  uint8_t* q_t;
  float* s_t;
};

struct NormColSmem {
  static constexpr int kIn = 0;                                  // 2 x 32 KB
  static constexpr int kEmit = 2 * kTileBytes;
  static constexpr int kBar = kEmit + TileEmit::kBytes;
  static constexpr int kBytes = kBar + 32;
  static constexpr int kAlloc = kBytes + 128;
};

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 2)
    norm_col_kernel(const __grid_constant__ CUtensorMap map_h, const NormColArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + NormColSmem::kBar;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + NormColSmem::kBar + 16);
  const int t = threadIdx.x, rb = t >> 4, cg = t & 15;
  const int num_tiles = a.tiles_r * a.tiles_c;
  if (t == 0) {
    mbar_init(bar0, 1);
    mbar_init(bar0 + 8, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    prefetch_tmap(&map_h);
  }
  __syncthreads();
  launch_dependents();
  grid_dependency_wait();
  // last rows first: they are the most recently written
  auto load = [&](int k, int b) {
    const int tile = num_tiles - 1 - k;
    mbar_arrive_expect_tx(bar0 + 8u * b, kTileBytes);
    tma_load_2d(sbase + NormColSmem::kIn + b * kTileBytes, &map_h, bar0 + 8u * b,
                (tile % a.tiles_c) * kTile, (a.tr0 + tile / a.tiles_c) * kTile);
  };
  int pend[2] = {-1, -1};
  if (t == 0) {
    for (int b = 0; b < 2; ++b) {
      const int k = blockIdx.x + b * gridDim.x;
      if (k < num_tiles) {
        load(k, b);
        pend[b] = 0;
      }
    }
  }
  int i = 0;
  for (int k = blockIdx.x; k < num_tiles; k += gridDim.x, ++i) {
    const int buf = i & 1;
    const int tile = num_tiles - 1 - k;
    const int tr = a.tr0 + tile / a.tiles_c, tc = tile % a.tiles_c;
    const int64_t r0 = static_cast<int64_t>(tr) * kTile + rb * 8;
    const int64_t c0 = static_cast<int64_t>(tc) * kTile + cg * 8;
    float g[8], rs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 0.0f;
    if (c0 < a.cols) load_gamma8(a.gamma, a.gamma_f32, c0, g);
#pragma unroll
    for (int p = 0; p < 8; ++p) rs[p] = r0 + p < a.rows ? __ldg(a.rstd + r0 + p) : 0.0f;
    const bool got = mbar_wait(bar0 + 8u * buf, (i >> 1) & 1, abort_flag, kErrTimeoutTma);
    if (!__syncthreads_and(got ? 1 : 0)) break;
    pend[buf] = -1;
    float y[8][8];
    const uint16_t* in = reinterpret_cast<const uint16_t*>(smem + NormColSmem::kIn + buf * kTileBytes);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      unpack8(ld16(in + (rb * 8 + p) * kTile + cg * 8), y[p]);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[p][j] = (y[p][j] * rs[p]) * g[j];
    }
    __syncthreads();   // the input buffer is free: fetch the tile after next
    if (t == 0) {
      const int next = k + 2 * gridDim.x;
      if (next < num_tiles) {
        load(next, buf);
        pend[buf] = ((i >> 1) + 1) & 1;
      }
    }
    const TileOut o{nullptr, nullptr, a.q_t, a.s_t, a.rows_pad, a.cols, tr, tc};
    emit_tile<false, true, POW2>(y, smem + NormColSmem::kEmit, o);
  }
  if (t == 0) drain_loads(bar0, pend, 2);
}

// ---------------------------------------------------------------- backward
struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const float* rstd;
  const void* gamma;
  int gamma_f32;
  const uint16_t* dres;       // may be null
  int64_t rows, cols;
  uint16_t* dh;
  float* part;                // [gridDim.x * groups][cols] partial dgamma
  int tpr;
};

// R rows x V chunks per thread and iteration; each group of tpr threads keeps
// its columns' dgamma sums in registers over all its rows. Long rows leave no
// registers for what the second half of an iteration needs: from V = 4 on dres
// is loaded only there, and with V = 8 dy and h are read again (from L2).
template <int V, int R>
__global__ void __launch_bounds__(512, 1) rmsnorm_bwd_kernel(const NormBwdArgs a) {
  constexpr bool kKeepRes = V <= 2, kKeep = V <= 4;
  __shared__ float part[2][R][16];
  launch_dependents();
  grid_dependency_wait();
  const int tpr = a.tpr;
  const int grp = threadIdx.x / tpr;
  const int t = threadIdx.x - grp * tpr;
  const int groups = blockDim.x / tpr;
  const int wpr = tpr >> 5;
  const int warp = threadIdx.x >> 5;
  const int chunks = static_cast<int>(a.cols >> 3);
  const float inv = __fdiv_rn(1.0f, static_cast<float>(a.cols));
  const int64_t per_block = static_cast<int64_t>(groups) * R;

  float acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.0f;

  int it = 0;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * per_block; b < a.rows;
       b += static_cast<int64_t>(gridDim.x) * per_block, ++it) {
    uint4 dy[R][V], h[R][V], dr[R][V];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float rs[R], dot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = b + r * groups + grp;
      const bool live = row < a.rows;
      rs[r] = live ? __ldg(a.rstd + row) : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = t + v * tpr;
        const int64_t at = row * a.cols + 8 * static_cast<int64_t>(c);
        const bool in = live && c < chunks;
        dy[r][v] = in ? (kKeep ? ld16_stream(a.dy + at) : ld16(a.dy + at)) : zero;
        h[r][v] = in ? (kKeep ? ld16_stream(a.h + at) : ld16(a.h + at)) : zero;
        if constexpr (kKeepRes) dr[r][v] = in && a.dres != nullptr ? ld16_stream(a.dres + at) : zero;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float g[8];
      const int c = t + v * tpr;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 0.0f;
      if (c < chunks) load_gamma8(a.gamma, a.gamma_f32, 8 * static_cast<int64_t>(c), g);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d[8], x[8];
        unpack8(dy[r][v], d);
        unpack8(h[r][v], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dx = d[j] * (x[j] * rs[r]);
          acc[v][j] += dx;
          dot[r] = fmaf(dx, g[j], dot[r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = warp_sum(dot[r]);
    if (wpr > 1) {
      float(*pt)[16] = part[it & 1];
      if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) pt[r][warp] = dot[r];
      }
      __syncthreads();   // the other buffer's readers are past the last one
#pragma unroll
      for (int r = 0; r < R; ++r) {
        dot[r] = 0.0f;
        for (int w = 0; w < wpr; ++w) dot[r] += pt[r][grp * wpr + w];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float g[8];
      const int c = t + v * tpr;
      if (c >= chunks) continue;
      load_gamma8(a.gamma, a.gamma_f32, 8 * static_cast<int64_t>(c), g);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t row = b + r * groups + grp;
        if (row >= a.rows) continue;
        const int64_t at = row * a.cols + 8 * static_cast<int64_t>(c);
        if constexpr (!kKeepRes) dr[r][v] = a.dres != nullptr ? ld16_stream(a.dres + at) : zero;
        if constexpr (!kKeep) {
          dy[r][v] = ld16_again(a.dy + at);
          h[r][v] = ld16_again(a.h + at);
        }
        float d[8], x[8], e[8];
        unpack8(dy[r][v], d);
        unpack8(h[r][v], x);
        unpack8(dr[r][v], e);
        const float m = dot[r] * inv;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          e[j] = fmaf(rs[r], fmaf(-(x[j] * rs[r]), m, d[j] * g[j]), e[j]);
        *reinterpret_cast<uint4*>(a.dh + at) =
            make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]),
                       pack_bf16(e[6], e[7]));
      }
    }
  }
  float* out = a.part + (static_cast<int64_t>(blockIdx.x) * groups + grp) * a.cols;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + v * tpr;
    if (c >= chunks) continue;
    float4* p = reinterpret_cast<float4*>(out + 8 * static_cast<int64_t>(c));
    p[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
    p[1] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
  }
}

// dgamma[c] = sum over the partial rows, in a fixed order (32 slices, then the
// slices one after another): the same bits for the same inputs every time.
__global__ void __launch_bounds__(1024)
    dgamma_reduce_kernel(const float* part, int64_t nparts, int64_t cols, float* dgamma) {
  __shared__ float sum[32][33];
  launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int64_t p = slice; p < nparts; p += 32) s += part[p * cols + c];
  sum[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < cols) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) r += sum[i][lane];
    dgamma[c] = r;
  }
}

}  // namespace layer
}  // namespace fp8bw
