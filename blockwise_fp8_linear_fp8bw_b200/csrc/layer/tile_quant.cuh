// tile_quant.cuh -- E4M3 quantisation of 128x128 tiles of fp32 values that a
// kernel holds in registers: row-wise codes with 1x128 scales and/or
// column-wise codes (transposed) with 128x1 scales, with the arithmetic and
// layouts of the quantisers. 256 threads; thread t owns the 8x8 sub-block of
// rows 8*(t/16) .. +7 and columns 8*(t%16) .. +7.
#pragma once

#include <cuda.h>

#include "../common.cuh"

namespace fp8bw {
namespace layer {

constexpr int kTile = 128;
constexpr int kTileThreads = 256;
constexpr int kTileBytes = kTile * kTile * 2;   // one bf16 tile

__device__ __forceinline__ uint8_t* align128(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 127) &
                                    ~static_cast<uintptr_t>(127));
}

// Encode 8 values (already multiplied by qscale) into 8 bytes.
__device__ __forceinline__ uint2 encode8(const float (&t)[8]) {
  return make_uint2(e4m3x2(t[0], t[1]) | (e4m3x2(t[2], t[3]) << 16),
                    e4m3x2(t[4], t[5]) | (e4m3x2(t[6], t[7]) << 16));
}

// Shared memory of emit_tile.
struct TileEmit {
  static constexpr int kT = 0;                          // transposed codes, 16 KB
  static constexpr int kRed = kT + kTile * kTile;       // 8 x 128 floats
  static constexpr int kColQ = kRed + 8 * kTile * 4;    // 128 floats
  static constexpr int kSRow = kColQ + kTile * 4;       // 128 floats
  static constexpr int kBytes = kSRow + kTile * 4;
};

// Where a tile's codes and scales go (row-wise or column-wise may be unused).
struct TileOut {
  uint8_t* q;          // [rows_pad][cols]
  float* s;            // [ceil(cols/128)][rows_pad]
  uint8_t* q_t;        // [cols][rows_pad]
  float* s_t;          // [ceil(rows_pad/128)][cols]
  int64_t rows, cols;  // rows = rows_pad, a multiple of 16; cols too
  int tr, tc;          // tile coordinates
};

// Byte offset in the transposed tile of the 8-byte unit of tokens 8u .. 8u+7
// of column k; units are xor-ed with the column block, so the 16 column blocks
// of a half-warp hit 16 different bank pairs.
__device__ __forceinline__ int emit_t_offset(int k, int u) {
  return k * kTile + ((u ^ (k >> 3)) & 15) * 8;
}

// All 256 threads call this with their 8x8 values; entries outside the tensor
// must be zero. Begins with the shared memory free (all threads past the
// previous use) and ends with a barrier after the last use.
// FENCE: the shared memory this block has written is about to be overwritten
// by bulk copies (issued after that barrier).
template <bool ROW, bool COL, bool POW2, bool FENCE = false>
__device__ __forceinline__ void emit_tile(const float (&y)[8][8], uint8_t* smem,
                                          const TileOut& o) {
  uint8_t* T = smem + TileEmit::kT;
  float(*red)[kTile] = reinterpret_cast<float(*)[kTile]>(smem + TileEmit::kRed);
  float* colq = reinterpret_cast<float*>(smem + TileEmit::kColQ);
  float* srow = reinterpret_cast<float*>(smem + TileEmit::kSRow);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, rb = t >> 4, cg = t & 15;
  const int64_t r0 = static_cast<int64_t>(o.tr) * kTile + rb * 8;
  const int64_t c0 = static_cast<int64_t>(o.tc) * kTile + cg * 8;
  const bool valid = r0 < o.rows && c0 < o.cols;

  if constexpr (COL) {
    // column maxima: 8 rows here, x2 across the half-warps, x8 warps below
    float cm[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cm[j] = fabsf(y[0][j]);
#pragma unroll
      for (int p = 1; p < 8; ++p) cm[j] = fmaxf(cm[j], fabsf(y[p][j]));
      cm[j] = fmaxf(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 16));
    }
    if (lane < 16) {
      float4* dst = reinterpret_cast<float4*>(&red[warp][cg * 8]);
      dst[0] = make_float4(cm[0], cm[1], cm[2], cm[3]);
      dst[1] = make_float4(cm[4], cm[5], cm[6], cm[7]);
    }
  }
  if constexpr (ROW) {
    // the 16 lanes of a half-warp share 8 rows; lane (cg & 7) computes the
    // scale of row (cg & 7)
    float mine = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float m = fabsf(y[p][0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(y[p][j]));
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      if ((cg & 7) == p) mine = m;
    }
    float qs, s;
    scale_of<POW2>(mine, qs, s);
    if (cg < 8) srow[rb * 8 + cg] = s;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float k = __shfl_sync(0xFFFFFFFFu, qs, (lane & 16) | p);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) fmul2(v[j], v[j + 1], y[p][j], y[p][j + 1], k, k);
      if (valid) *reinterpret_cast<uint2*>(o.q + (r0 + p) * o.cols + c0) = encode8(v);
    }
  }
  if constexpr (COL) {
    __syncthreads();
    if (t < kTile) {
      float m = red[0][t];
#pragma unroll
      for (int w = 1; w < kTileThreads / 32; ++w) m = fmaxf(m, red[w][t]);
      float qs, s;
      scale_of<POW2>(m, qs, s);
      colq[t] = qs;
      const int64_t col = static_cast<int64_t>(o.tc) * kTile + t;
      if (col < o.cols) o.s_t[static_cast<int64_t>(o.tr) * o.cols + col] = s;
    }
    __syncthreads();
    const float4 q0 = *reinterpret_cast<const float4*>(&colq[cg * 8]);
    const float4 q1 = *reinterpret_cast<const float4*>(&colq[cg * 8 + 4]);
    const float qv[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v[8];
#pragma unroll
      for (int p = 0; p < 8; p += 2) fmul2(v[p], v[p + 1], y[p][j], y[p + 1][j], qv[j], qv[j]);
      *reinterpret_cast<uint2*>(T + emit_t_offset(cg * 8 + j, rb)) = encode8(v);
    }
  }
  __syncthreads();
  if constexpr (ROW) {
    if (t < kTile / 4) {
      const int64_t row = static_cast<int64_t>(o.tr) * kTile + t * 4;
      if (row < o.rows)
        *reinterpret_cast<float4*>(o.s + static_cast<int64_t>(o.tc) * o.rows + row) =
            *reinterpret_cast<const float4*>(&srow[t * 4]);
    }
  }
  if constexpr (COL) {
    // tile column k is 128 contiguous tokens of row tc*128 + k of q_t
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int idx = it * kTileThreads + t;
      const int kk = idx >> 3, ch = idx & 7;
      const int64_t col = static_cast<int64_t>(o.tc) * kTile + kk;
      const int64_t tok = static_cast<int64_t>(o.tr) * kTile + ch * 16;
      if (col < o.cols && tok < o.rows) {
        const uint2 lo = *reinterpret_cast<const uint2*>(T + emit_t_offset(kk, 2 * ch));
        const uint2 hi = *reinterpret_cast<const uint2*>(T + emit_t_offset(kk, 2 * ch + 1));
        *reinterpret_cast<uint4*>(o.q_t + col * o.rows + tok) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
  if constexpr (FENCE) fence_proxy_async_smem();
  __syncthreads();
}

// After an early exit: wait (bounded) for the loads still in flight before the
// shared memory is released. pend[b]: parity of a load nobody waited for, or -1.
__device__ __forceinline__ void drain_loads(uint32_t bar0, const int* pend, int n) {
  for (int b = 0; b < n; ++b) {
    if (pend[b] < 0) continue;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar0 + 8u * b, static_cast<uint32_t>(pend[b])) &&
           globaltimer_ns() - t0 < kWaitLimitNs) {
    }
  }
}

}  // namespace layer
}  // namespace fp8bw
