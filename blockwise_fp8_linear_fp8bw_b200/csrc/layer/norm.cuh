// norm.cuh -- residual addition + root-mean-square norm whose output leaves as
// E4M3 codes, and its backward pass (sm_100a, HBM-bound).
//
//   h    = bf16(x + residual)                (h = x without a residual)
//   rstd = 1 / sqrt(mean_c h^2 + eps)        fp32
//   y    = h * rstd * gamma                  fp32
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
// second pass over h in 128 x 64 tiles, last rows first, while the end of h is
// still in L2.
#pragma once

#include "../common.cuh"
#include "tile_quant.cuh"

namespace fp8bw {
namespace layer {

// ---------------------------------------------------------------- helpers
__device__ __forceinline__ uint4 ld16(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// Inputs may come from the kernel before this one, so no load may move above
// grid_dependency_wait(): they are volatile (that keeps their order with the
// wait), not loads of constant memory.

// Read once, not needed again: keep it from displacing what is re-read from L2.
__device__ __forceinline__ uint4 ld16_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A load of its own: the compiler neither merges it with another of the same
// address (whose registers would then have to live until here) nor holds it back
// behind a store.
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
    const float* p = static_cast<const float*>(gamma) + c;
    const uint4 a = ld16_again(p), b = ld16_again(p + 4);
    g[0] = __uint_as_float(a.x), g[1] = __uint_as_float(a.y);
    g[2] = __uint_as_float(a.z), g[3] = __uint_as_float(a.w);
    g[4] = __uint_as_float(b.x), g[5] = __uint_as_float(b.y);
    g[6] = __uint_as_float(b.z), g[7] = __uint_as_float(b.w);
  } else {
    unpack8(ld16_again(static_cast<const uint16_t*>(gamma) + c), g);
  }
}

// One of them.
__device__ __forceinline__ float load_gamma(const void* gamma, int is_f32, int64_t c) {
  return is_f32 ? static_cast<const float*>(gamma)[c]
                : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(gamma)[c])
                                  << 16);
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
  int64_t rows, rows_pad, cols;
  double inv_cols;
  float eps;
  uint16_t* h;                // written when there is a residual
  float* rstd;                // may be null
  uint16_t* y;                // bf16 output, may be null
  uint8_t* q;                 // row-wise codes, may be null
  float* s;                   // their scales [ceil(cols/128)][rows_pad]
  int tpr;                    // threads per row, a multiple of 32
};

constexpr int kNormMaxWarps = 32;

// 1 / sqrt(sum / cols + eps), rounded once: its error is in every value of the row.
// The approximate root and one Newton step in 64 bits (not from zero or infinity).
__device__ __forceinline__ float rsqrt_of_mean(float sum, double inv_cols, float eps) {
  const double x = fma(static_cast<double>(sum), inv_cols, static_cast<double>(eps));
  const float r = rsqrtf(static_cast<float>(x));
  const double d = r, n = d * fma(-0.5 * x * d, d, 1.5);
  return r > 0.0f && r < 1e30f ? static_cast<float>(n) : r;
}

// Element-wise bf16 sums of two packed vectors, each rounded once.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hadd2_rn(*reinterpret_cast<__nv_bfloat162*>(&a),
                                      *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint4 add_bf16x8(const uint4& a, const uint4& b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z),
                    add_bf16x2(a.w, b.w));
}

// R rows x V chunks of 8 columns per thread; blockDim = groups x tpr, R rows each.
// FULL: the row is exactly V x tpr chunks. h * gamma and the groups' maxima of
// it are formed before rstd is known, so all that is left after the row sum is
// one product per element: codes are E4M3(h gamma * (rstd * qscale)).
template <int V, int R, bool FULL, bool POW2>
__global__ void __launch_bounds__(V * R == 1 ? 1024 : 512)
    rmsnorm_row_kernel(const NormArgs a) {
  constexpr int N = V * R;                     // item i: chunk i / R of row i % R
  __shared__ float part[kNormMaxWarps][R];
  launch_dependents();
  grid_dependency_wait();
  const int tpr = a.tpr;
  const int grp = threadIdx.x / tpr;
  const int t = threadIdx.x - grp * tpr;
  const int groups = blockDim.x / tpr;
  const int lane = threadIdx.x & 31;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * groups + grp) * R;
  const int chunks = static_cast<int>(a.cols >> 3);
  const int64_t base = row0 * a.cols + 8 * t;
  auto has = [&](int i) { return FULL || t + i / R * tpr < chunks; };
  auto live = [&](int i) { return row0 + i % R < a.rows; };
  auto at = [&](int i) { return base + i % R * a.cols + 8 * (i / R * tpr); };

  uint4 h[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    h[i] = live(i) && has(i) ? ld16_stream(a.x + at(i)) : make_uint4(0u, 0u, 0u, 0u);
  if (a.residual != nullptr) {
    uint4 r[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      r[i] = live(i) && has(i) ? ld16_stream(a.residual + at(i)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      h[i] = add_bf16x8(h[i], r[i]);
      if (live(i) && has(i)) *reinterpret_cast<uint4*>(a.h + at(i)) = h[i];
    }
  }

  float ss[R], y[N][8], m[N];
#pragma unroll
  for (int r = 0; r < R; ++r) ss[r] = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float g[8];
    if (has(v * R)) load_gamma8(a.gamma, a.gamma_f32, 8 * static_cast<int64_t>(t + v * tpr), g);
    else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 0.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = v * R + r;
      unpack8(h[i], y[i]);
      m[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        ss[r] = fmaf(y[i][j], y[i][j], ss[r]);
        ss[r] = fmaf(y[i][j + 1], y[i][j + 1], ss[r]);
        fmul2(y[i][j], y[i][j + 1], y[i][j], y[i][j + 1], g[j], g[j + 1]);
        m[i] = max3_abs(m[i], y[i][j], y[i][j + 1]);
      }
    }
  }
  // group maxima over the 16 lanes of a half-warp: lanes halve the groups they
  // hold as they exchange, so that each ends up with one of the N
#pragma unroll
  for (int half = N / 2, bit = 8; bit >= 1; bit >>= 1) {
    if (half >= 1) {
      const bool up = (lane & bit) != 0;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float send = up ? m[i] : m[i + half];
        const float keep = up ? m[i + half] : m[i];
        m[i] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, send, bit));
      }
      half >>= 1;
    } else {
      m[0] = fmaxf(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], bit));
    }
  }
  constexpr int kShare = 16 / N;               // lanes that hold the same group
  const int mine = (lane & 15) / kShare;       // which one

#pragma unroll
  for (int r = 0; r < R; ++r) ss[r] = warp_sum(ss[r]);
  const int wpr = tpr >> 5;
  if (wpr > 1) {
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) part[threadIdx.x >> 5][r] = ss[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) ss[r] = 0.0f;
    for (int w = 0; w < wpr; ++w) {
#pragma unroll
      for (int r = 0; r < R; ++r) ss[r] += part[grp * wpr + w][r];
    }
  }
  float rstd[R], my_rstd = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    rstd[r] = rsqrt_of_mean(ss[r], a.inv_cols, a.eps);
    if (live(r) && t == 0 && a.rstd != nullptr) a.rstd[row0 + r] = rstd[r];
    if (mine % R == r) my_rstd = rstd[r];
  }
  const int64_t first = (t & ~15) + mine / R * tpr;   // first chunk of this lane's group
  const bool group = FULL || first < chunks;

  // (h gamma) rstd, the order above, may leave fp32's range where (h rstd) gamma does
  // not. What is outside of [2^-100, 2^120] on the way is done over below, from h once
  // more and in the formula's order. (Zeros only where rstd could bring a product
  // below 2^-150 back.)
  auto outside = [](float v, float rs) {
    return !(v >= 0x1p-100f && v <= 0x1p120f) && !(v == 0.0f && rs <= 1024.0f);
  };
  uint32_t low = 0u;                           // items with such a value of y
  if (a.y != nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!live(i) || !has(i)) continue;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (outside(fabsf(y[i][j]), rstd[i % R])) low |= 1u << i;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_bf16(y[i][2 * j] * rstd[i % R], y[i][2 * j + 1] * rstd[i % R]);
      *reinterpret_cast<uint4*>(a.y + at(i)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  bool odd = false;                            // a group's codes
  if (a.q != nullptr) {
    const float top = m[0] * my_rstd;
    odd = group && row0 + mine % R < a.rows && (outside(m[0], my_rstd) || !(top <= 0x1p120f));
    float qs, s;
    scale_near<POW2>(top, qs, s);
    float f = qs * my_rstd;
    if constexpr (!POW2) {
      // rstd cancels: 448 / max|h gamma|, three roundings fewer (not where a scale of
      // 1 stands for none)
      const float d = near_448_over(m[0]);
      if (isfinite(d) && !(qs == 1.0f && s == 1.0f)) f = d;
    }
    if ((lane & (kShare - 1)) == 0 && row0 + mine % R < a.rows_pad && group && !odd)
      a.s[(first >> 4) * a.rows_pad + row0 + mine % R] = s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float k = __shfl_sync(0xFFFFFFFFu, f, (lane & 16) | (i * kShare));
      // (a padding row is zero whatever its factor is: without eps its rstd is infinite)
      uint2 w = make_uint2(0u, 0u);
      if (live(i)) {
        w.x = encode4(y[i][0], y[i][1], y[i][2], y[i][3], k);
        w.y = encode4(y[i][4], y[i][5], y[i][6], y[i][7], k);
      }
      if (row0 + i % R < a.rows_pad && has(i)) *reinterpret_cast<uint2*>(a.q + at(i)) = w;
    }
  }
  if (!__any_sync(0xFFFFFFFFu, odd || low != 0u)) return;
  // (each thread over what it wrote itself)
#pragma unroll 1
  for (int i = 0; i < N; ++i) {
    const int from = (lane & 16) | (i * kShare);
    const float rs = __shfl_sync(0xFFFFFFFFu, my_rstd, from);
    const bool codes = __shfl_sync(0xFFFFFFFFu, odd, from) != 0 && has(i);
    float v[8], most = 0.0f;
    if (codes || (low >> i & 1u)) {
      float g[8];
      uint4 w = ld16_again(a.x + at(i));
      if (a.residual != nullptr) w = add_bf16x8(w, ld16_again(a.residual + at(i)));
      unpack8(w, v);
      load_gamma8(a.gamma, a.gamma_f32, 8 * static_cast<int64_t>(t + i / R * tpr), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = __fmul_rn(__fmul_rn(v[j], rs), g[j]);
        most = max3_abs(most, v[j], v[j]);
      }
      if (low >> i & 1u)
        *reinterpret_cast<uint4*>(a.y + at(i)) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                       pack_bf16(v[6], v[7]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (!codes) continue;
    float qs, s;
    scale_near<POW2>(most, qs, s);
    *reinterpret_cast<uint2*>(a.q + at(i)) =
        make_uint2(encode4(v[0], v[1], v[2], v[3], qs), encode4(v[4], v[5], v[6], v[7], qs));
    if ((lane & 15) == 0) a.s[((t + i / R * tpr) >> 4) * a.rows_pad + row0 + i % R] = s;
  }
}

// ---------------------------------------------------------------- forward, column-wise
// y of a 128 x 64 tile of h, from the rows' rstd, to column-wise codes. A block does
// one tile and four blocks share an SM: a tile is a chain of loads and barriers, and
// the other blocks work meanwhile. (16384 x 2048, both passes: 59.2 us. When it was
// 61, steps of one 512-thread block per SM over 128 x 128 tiles with a TMA ring took
// 63 and persistent blocks that copy the next tile ahead 66.)
struct NormColArgs {
  const uint16_t* h;
  const float* rstd;
  const void* gamma;
  int gamma_f32;
  int64_t rows, rows_pad, cols;
  int tiles_r, tiles_c;
  uint8_t* q_t;
  float* s_t;
};

template <bool POW2>
__global__ void __launch_bounds__(kColThreads, 4) norm_col_kernel(const NormColArgs a) {
  __shared__ ColumnsSmem sm;
  launch_dependents();
  grid_dependency_wait();
  const int t = threadIdx.x, rb = t >> 4, cb = t & 15;
  // last rows first: they are the most recently written, and still in L2
  const int tile = a.tiles_r * a.tiles_c - 1 - static_cast<int>(blockIdx.x);
  const int tr = tile / a.tiles_c, tc = tile % a.tiles_c;
  const int64_t r0 = static_cast<int64_t>(tr) * kTile + rb * 8;
  const int64_t c0 = static_cast<int64_t>(tc) * kColTile + cb * 4;
  // h * rstd; the norm weight joins a column's scale
  uint2 w[8];
  float rs[8];
  const uint16_t* h = a.h + r0 * a.cols + c0;
  if (static_cast<int64_t>(tr + 1) * kTile <= a.rows &&
      static_cast<int64_t>(tc + 1) * kColTile <= a.cols) {
    const float4 ra = reinterpret_cast<const float4*>(a.rstd + r0)[0];
    const float4 rc = reinterpret_cast<const float4*>(a.rstd + r0)[1];
    rs[0] = ra.x, rs[1] = ra.y, rs[2] = ra.z, rs[3] = ra.w;
    rs[4] = rc.x, rs[5] = rc.y, rs[6] = rc.z, rs[7] = rc.w;
#pragma unroll
    for (int p = 0; p < 8; ++p, h += a.cols) w[p] = *reinterpret_cast<const uint2*>(h);
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p, h += a.cols) {
      const bool in = c0 < a.cols && r0 + p < a.rows;
      w[p] = in ? *reinterpret_cast<const uint2*>(h) : make_uint2(0u, 0u);
      rs[p] = in ? a.rstd[r0 + p] : 0.0f;
    }
  }
  float y[8][4], m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    fmul2(y[p][0], y[p][1], bf16_lo(w[p].x), bf16_hi(w[p].x), rs[p], rs[p]);
    fmul2(y[p][2], y[p][3], bf16_lo(w[p].y), bf16_hi(w[p].y), rs[p], rs[p]);
    if (p & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = max3_abs(m[j], y[p - 1][j], y[p][j]);
    }
  }
  emit_columns<POW2>(sm, y, m, tr, tc, a.rows_pad, a.cols, a.q_t, a.s_t,
                     static_cast<int>(min(max(a.rows - r0, int64_t(0)), int64_t(8))),
                     [&](int64_t c) { return load_gamma(a.gamma, a.gamma_f32, c); });
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
  float* part;                // [gridDim.x][cols] partial dgamma
  int tpr;
};

// R rows x V chunks per thread and iteration; each group of tpr threads keeps
// its columns' dgamma sums in registers over all its rows. With
//   s = rstd * sum_c dy gamma h   (so that mean_c(g xh) = s / cols)
// a row is  dh = rstd (dy gamma) - (rstd^2 s / cols) h + dres: three products
// per element before the row sum and three after it. The next iteration's rows are
// loaded before this one's are worked on (16384 x 2048: 47 us; with twice the rows
// per iteration and nothing ahead 50; through a shared-memory ring with a warp per
// row 61). Long rows leave no registers for that, nor for what the second half of
// an iteration needs: from V = 4 on dres and gamma are loaded again there, and
// with V = 8 dy and h too (from L2).
template <int V, int R>
__global__ void __launch_bounds__(512, 1) rmsnorm_bwd_kernel(const NormBwdArgs a) {
  constexpr bool kKeepRes = V <= 2, kKeep = V <= 4, kAhead = V * R <= 2;
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
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto has = [&](int v) { return t + v * tpr < chunks; };
  auto col = [&](int v) { return 8 * static_cast<int64_t>(t + v * tpr); };

  float acc[V][8], gamma[kKeepRes ? V : 1][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.0f;
  auto load_gamma = [&](int v, float (&g)[8]) {
    if (has(v)) {
      load_gamma8(a.gamma, a.gamma_f32, col(v), g);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 0.0f;
    }
  };
  if constexpr (kKeepRes) {
#pragma unroll
    for (int v = 0; v < V; ++v) load_gamma(v, gamma[v]);
  }

  int it = 0;
  uint4 dy[R][V], h[R][V], dr[R][V];
  float rs[R];
  auto load_rows = [&](int64_t b, uint4 (&dy)[R][V], uint4 (&h)[R][V], uint4 (&dr)[R][V],
                       float (&rs)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = b + r * groups + grp;
      const bool live = row < a.rows;
      rs[r] = live ? a.rstd[row] : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t at = row * a.cols + col(v);
        const bool in = live && has(v);
        dy[r][v] = in ? (kKeep ? ld16_stream(a.dy + at) : ld16(a.dy + at)) : zero;
        h[r][v] = in ? (kKeep ? ld16_stream(a.h + at) : ld16(a.h + at)) : zero;
        if constexpr (kKeepRes) dr[r][v] = in && a.dres != nullptr ? ld16_stream(a.dres + at) : zero;
      }
    }
  };
  const int64_t bstep = static_cast<int64_t>(gridDim.x) * per_block;
  int64_t b = static_cast<int64_t>(blockIdx.x) * per_block;
  if (b < a.rows) load_rows(b, dy, h, dr, rs);
  for (; b < a.rows; b += bstep, ++it) {
    uint4 ndy[R][V], nh[R][V], ndr[R][V];
    float nrs[R], dot[R];
    if constexpr (kAhead) {
      if (b + bstep < a.rows) load_rows(b + bstep, ndy, nh, ndr, nrs);
    }
    float d0[R], d1[R];
#pragma unroll
    for (int r = 0; r < R; ++r) d0[r] = d1[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (!kKeepRes) load_gamma(v, gamma[0]);
      const float(&g)[8] = gamma[kKeepRes ? v : 0];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d[8], x[8];
        unpack8(dy[r][v], d);
        unpack8(h[r][v], x);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float p0, p1;
          fmul2(p0, p1, d[j], d[j + 1], x[j], x[j + 1]);
          ffma2(acc[v][j], acc[v][j + 1], p0, p1, rs[r], rs[r]);
          ffma2(d0[r], d1[r], p0, p1, g[j], g[j + 1]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = warp_sum(d0[r] + d1[r]);
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
      if (!has(v)) continue;
      if constexpr (!kKeepRes) load_gamma(v, gamma[0]);
      const float(&g)[8] = gamma[kKeepRes ? v : 0];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t row = b + r * groups + grp;
        if (row >= a.rows) continue;
        const int64_t at = row * a.cols + col(v);
        if constexpr (!kKeepRes) dr[r][v] = a.dres != nullptr ? ld16_stream(a.dres + at) : zero;
        if constexpr (!kKeep) {
          dy[r][v] = ld16_again(a.dy + at);
          h[r][v] = ld16_again(a.h + at);
        }
        float d[8], x[8], e[8];
        unpack8(dy[r][v], d);
        unpack8(h[r][v], x);
        unpack8(dr[r][v], e);
        const float k = -(rs[r] * rs[r]) * (rs[r] * dot[r] * inv);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float p0, p1;
          fmul2(p0, p1, d[j], d[j + 1], g[j], g[j + 1]);
          ffma2(e[j], e[j + 1], p0, p1, rs[r], rs[r]);
          ffma2(e[j], e[j + 1], x[j], x[j + 1], k, k);
          w[j >> 1] = pack_bf16(e[j], e[j + 1]);
        }
        *reinterpret_cast<uint4*>(a.dh + at) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        rs[r] = nrs[r];
#pragma unroll
        for (int v = 0; v < V; ++v) dy[r][v] = ndy[r][v], h[r][v] = nh[r][v], dr[r][v] = ndr[r][v];
      }
    } else if (b + bstep < a.rows) {
      load_rows(b + bstep, dy, h, dr, rs);
    }
  }
  if constexpr (V == 1) {
    // the groups' sums, one after another (blocks of several groups have up to 128
    // threads)
    if (groups > 1) {
      __shared__ float4 sums[128][2];
      if (grp > 0) {
        sums[threadIdx.x][0] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
        sums[threadIdx.x][1] = make_float4(acc[0][4], acc[0][5], acc[0][6], acc[0][7]);
      }
      __syncthreads();
      if (grp > 0) return;
      for (int g = 1; g < groups; ++g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 s = sums[g * tpr + t][i];
          acc[0][4 * i] += s.x, acc[0][4 * i + 1] += s.y;
          acc[0][4 * i + 2] += s.z, acc[0][4 * i + 3] += s.w;
        }
      }
    }
  }
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + v * tpr;
    if (c >= chunks) continue;
    float4* p = reinterpret_cast<float4*>(out + 8 * static_cast<int64_t>(c));
    p[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
    p[1] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
  }
}

// dgamma[c] = sum over the partial rows, in a fixed order (slices, a warp's, then the
// warps one after another): the same bits for the same inputs every time. A block
// takes C columns in 1024 / C slices of the rows: few columns for narrow norms, whose
// blocks would otherwise be few and their slices long.
template <int C>
__global__ void __launch_bounds__(1024)
    dgamma_reduce_kernel(const float* part, int64_t nparts, int64_t cols, float* dgamma) {
  __shared__ float sum[32][C + 1];
  launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * C + lane % C;
  float s = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int64_t p = threadIdx.x / C; p < nparts; p += 1024 / C) s += part[p * cols + c];
#pragma unroll
  for (int o = C; o < 32; o *= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane < C) sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && lane < C && c < cols) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) r += sum[i][lane];
    dgamma[c] = r;
  }
}

}  // namespace layer
}  // namespace fp8bw
