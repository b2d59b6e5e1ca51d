// swiglu.cuh -- the SiLU-gated product of a fused gate/up projection and its
// backward pass, leaving as E4M3 codes (sm_100a, HBM-bound).
//
//   [gate | up] = gu[rows, 2f],  sg = 1 / (1 + exp(-gate))
//   a     = gate * sg * up                                  [rows, f]
//   dgate = da * up * sg * (1 + gate * (1 - sg))
//   dup   = da * gate * sg                                  d = [dgate | dup]
// computed in fp32 and rounded once, to E4M3: neither a nor d exists in bf16.
// The layouts are the quantisers' (row-wise codes for the next GEMM,
// column-wise transposed codes for the weight-gradient GEMM).
#pragma once

#include "norm.cuh"
#include "tile_quant.cuh"

namespace fp8bw {
namespace layer {

// 1 / (1 + exp(-x)) of two bf16 values by the approximate exponential and reciprocal
// (packed arithmetic where the instruction exists). log2(e) is taken as H + L with H of
// 16 bits: x H is exact, and what x L leaves out, at most 4.4e-4 of exp(-x), is added
// to first order. Relative error in units of 2^-24, rms and largest, over the bf16 x in
// [-4, 4]: 0.9 and 3.0; in [-80, 0] 1.1 and 3.4 (by the rounded product x log2(e) 5 and
// 14 down to -20, 28 and 55 down to -80; by expf and an IEEE quotient 0.8 and 2.3).
// Results that would be subnormal are 0, so below -87 the quotient is 0 (its value there
// is under 2^-125); at -inf it is 0, so that x * sigmoid(x) is NaN as the formula says.
// (Of NaN it is 1; what it multiplies is NaN.)
__device__ __forceinline__ void sigmoid2(float x0, float x1, float& s0, float& s1) {
  constexpr double kLog2e = 1.4426950408889634, kH = 47274.0 / 32768.0;
  constexpr float h = static_cast<float>(kH);
  constexpr float k = static_cast<float>(-(kLog2e - kH) * 0.6931471805599453 / kH);
  float p0, p1, e0, e1, t0 = 1.0f, t1 = 1.0f, d0 = 1.0f, d1 = 1.0f;
  fmul2(p0, p1, x0, x1, h, h);
  p0 = fminf(p0, 150.0f);                     // (infinity times 0 is NaN below)
  p1 = fminf(p1, 150.0f);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(-p0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(-p1));
  ffma2(t0, t1, p0, p1, k, k);
  ffma2(d0, d1, e0, e1, t0, t1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(d0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(d1));
}

// y = gate * sigmoid(gate) * up, two elements (in this order nothing overflows
// that the result does not).
__device__ __forceinline__ void glu2(const float* g, const float* u, float* y) {
  float s0, s1, w0, w1;
  sigmoid2(g[0], g[1], s0, s1);
  fmul2(w0, w1, g[0], g[1], s0, s1);
  fmul2(y[0], y[1], w0, w1, u[0], u[1]);
}

// Two elements of the backward pass.
__device__ __forceinline__ void glu_grad2(const float* g, const float* u, const float* d,
                                          float* dgate, float* dup) {
  float s0, s1, w0, w1, c0 = 1.0f, c1 = 1.0f;
  sigmoid2(g[0], g[1], s0, s1);
  fmul2(w0, w1, d[0], d[1], s0, s1);
  fmul2(dup[0], dup[1], w0, w1, g[0], g[1]);
  fmul2(w0, w1, w0, w1, u[0], u[1]);
  ffma2(c0, c1, s0, s1, -1.0f, -1.0f);          // 1 - sg
  float t0 = 1.0f, t1 = 1.0f;
  ffma2(t0, t1, g[0], g[1], c0, c1);            // 1 + gate (1 - sg)
  fmul2(dgate[0], dgate[1], w0, w1, t0, t1);
}

// ---------------------------------------------------------------- row-wise, or few tiles
// BWD: d = [dgate | dup], else a. The row-wise part of an output takes a half-warp
// per row and 1x128 group (a block: 16 rows of one group, so its scales are one
// 64-byte run), the column-wise part a block per 128 x 64 tile; both in one launch,
// each from inputs of its own (read twice, from L2). For no more than a tile per SM
// that is quicker than the kernels below (us, here and there: 1 x 6144 2.1 and 6.7,
// 100 x 1360 3.9 and 6.8, 1000 x 2048 6.3 and 7.1, 1000 x 4096 10.6 and 7.7; backward
// 1 x 6144 2.4 and 5.6, 100 x 1360 4.3 and 5.3, 300 x 2048 5.5 and 6.0, 777 x 1360
// 7.5 and 7.0).
struct GluFewArgs {
  const uint16_t* gu;
  const uint16_t* da;       // BWD
  int64_t rows, f;
  CodesOut out;
  int row_blocks;           // the first ones; the others take tiles
  int tiles_c;
};

// The input columns of output column c of BWD.
__device__ __forceinline__ int64_t glu_source(int64_t c, int64_t f) { return c >= f ? c - f : c; }

// Rows 16 i .. 16 i + 15 of a 1x128 group, by 256 threads.
template <bool POW2, bool BWD>
__device__ __forceinline__ void glu_rows(const GluFewArgs& a, int64_t i, int64_t group) {
  const int t = threadIdx.x;
  const int64_t row = i * 16 + (t >> 4), c = group * kTile + (t & 15) * 8;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = 0.0f;
  if (row < a.rows && c < a.out.cols) {
    const int64_t src = BWD ? glu_source(c, a.f) : c;
    const uint16_t* p = a.gu + row * 2 * a.f + src;
    const uint4 wg = ld16_stream(p), wu = ld16_stream(p + a.f);
    float g[8], u[8];
    unpack8(wg, g);
    unpack8(wu, u);
    if constexpr (BWD) {
      float d[8], dg[8], du[8];
      unpack8(ld16_stream(a.da + row * a.f + src), d);
#pragma unroll
      for (int j = 0; j < 8; j += 2) glu_grad2(g + j, u + j, d + j, dg + j, du + j);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = c >= a.f ? du[j] : dg[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; j += 2) glu2(g + j, u + j, y + j);
    }
  }
  float m = max3_abs(max3_abs(0.0f, y[0], y[1]), y[2], y[3]);
  m = max3_abs(max3_abs(m, y[4], y[5]), y[6], y[7]);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float qs, s;
  scale_near<POW2>(m, qs, s);
  if (c < a.out.cols)
    *reinterpret_cast<uint2*>(a.out.q + row * a.out.cols + c) =
        make_uint2(encode4(y[0], y[1], y[2], y[3], qs), encode4(y[4], y[5], y[6], y[7], qs));
  if ((t & 15) == 0) a.out.s[group * a.out.rows + row] = s;
}

template <bool POW2>
__global__ void __launch_bounds__(kColThreads) swiglu_row_kernel(const GluFewArgs a) {
  launch_dependents();
  grid_dependency_wait();
  glu_rows<POW2, false>(a, blockIdx.x, blockIdx.y);
}

// (forward, five blocks per SM: 1000 x 1024 5.6 us, with four 6.0)
template <bool POW2, bool BWD>
__global__ void __launch_bounds__(kColThreads, BWD ? 4 : 5)
    swiglu_few_kernel(const GluFewArgs a) {
  __shared__ ColumnsSmem sm;
  launch_dependents();
  grid_dependency_wait();
  const int t = threadIdx.x;
  if (static_cast<int>(blockIdx.x) < a.row_blocks) {
    const int rb = static_cast<int>(a.out.rows / 16);
    glu_rows<POW2, BWD>(a, blockIdx.x % rb, blockIdx.x / rb);
    return;
  }
  const int tile = static_cast<int>(blockIdx.x) - a.row_blocks;
  const int tr = tile / a.tiles_c, tc = tile % a.tiles_c;
  const int64_t r0 = static_cast<int64_t>(tr) * kTile + (t >> 4) * 8;
  const int64_t c = static_cast<int64_t>(tc) * kColTile + (t & 15) * 4;
  const int64_t src = BWD ? glu_source(c, a.f) : c;
  float y[8][4], m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int p = 0; p < 8; ++p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[p][j] = 0.0f;
    if (r0 + p < a.rows && c < a.out.cols) {
      const uint16_t* gp = a.gu + (r0 + p) * 2 * a.f + src;
      const uint2 wg = *reinterpret_cast<const uint2*>(gp);
      const uint2 wu = *reinterpret_cast<const uint2*>(gp + a.f);
      const float g[4] = {bf16_lo(wg.x), bf16_hi(wg.x), bf16_lo(wg.y), bf16_hi(wg.y)};
      const float u[4] = {bf16_lo(wu.x), bf16_hi(wu.x), bf16_lo(wu.y), bf16_hi(wu.y)};
      if constexpr (BWD) {
        const uint2 wd = *reinterpret_cast<const uint2*>(a.da + (r0 + p) * a.f + src);
        const float d[4] = {bf16_lo(wd.x), bf16_hi(wd.x), bf16_lo(wd.y), bf16_hi(wd.y)};
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          float dg[2], du[2];
          glu_grad2(g + j, u + j, d + j, dg, du);
          y[p][j] = c >= a.f ? du[0] : dg[0];
          y[p][j + 1] = c >= a.f ? du[1] : dg[1];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2) glu2(g + j, u + j, &y[p][j]);
      }
    }
    if (p & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = max3_abs(m[j], y[p - 1][j], y[p][j]);
    }
  }
  emit_columns<POW2>(sm, y, m, tr, tc, a.out.rows, a.out.cols, a.out.q_t, a.out.s_t, 8,
                     NoGain());
}

// ---------------------------------------------------------------- 128x128 tiles
struct GluTileArgs {
  int tiles_r, tiles_c;     // of the inputs' [rows, f]
  CodesOut out;
};

// Forward: two tiles per step, half the columns apart, so that the barriers of a
// step stand beside twice the work (16384 x 6144: 111 us, 5.5 TB/s; one
// tile per step, in two blocks per SM, took 6% longer).
constexpr int kGluFwdSlots = 6;
using GluFwdRing = TileRing<4, kGluFwdSlots>;      // gate, up, twice
struct GluFwdSmem {
  static constexpr int kEmit = (GluFwdRing::kBytes + 127) / 128 * 128;
  static constexpr int kAlloc = kEmit + TileEmit<2, false>::kBytes + 128;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 1)
    swiglu_tile_kernel(const __grid_constant__ CUtensorMap map_g,
                       const __grid_constant__ CUtensorMap map_u, const GluTileArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const int half = (a.tiles_c + 1) / 2;
  const int count = tiles_of_block(a.tiles_r * half);
  GluFwdRing ring(smem, count);
  if (threadIdx.x == 0) {
    ring.init();
    prefetch_tmap(&map_g);
    prefetch_tmap(&map_u);
  }
  TileEmit<2, POW2>::init(smem + GluFwdSmem::kEmit);
  __syncthreads();
  launch_dependents();
  grid_dependency_wait();
  auto load = [&](int i, int n, uint32_t dst, uint32_t bar) {
    const int tile = static_cast<int>(blockIdx.x + i * gridDim.x);
    // (a second tile past the end reads zeros)
    const int tc = tile % half + (n >= 2 ? half : 0);
    tma_load_2d(dst, n % 2 == 0 ? &map_g : &map_u, bar, tc * kTile, (tile / half) * kTile);
  };
  if (threadIdx.x == 0) ring.fill(kGluFwdSlots, load);
  TileEmit<2, POW2> emit(smem + GluFwdSmem::kEmit, a.out);
  for (int i = 0; i < count; ++i) {
    const int tile = static_cast<int>(blockIdx.x + i * gridDim.x);
    float y[2][8][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint8_t* gate = ring.next();
      const uint8_t* up = ring.next();
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        float g[4], u[4];
        read4(gate, p, g);
        read4(up, p, u);
#pragma unroll
        for (int j = 0; j < 4; j += 2) glu2(g + j, u + j, &y[n][p][j]);
      }
    }
    emit.step(y, tile / half, {tile % half, tile % half + half}, [&] {
      if (threadIdx.x == 0) ring.fill(4, load);
    });
  }
  emit.finish();
  if (threadIdx.x == 0) ring.drain();
}

// Backward, f a multiple of 128 (so that the groups of d do not straddle its
// two halves): gate, up and da tiles in, a dgate and a dup tile out (16384 x 6144:
// 171 us, 6.0 TB/s).
constexpr int kGluBwdSlots = 6;
using GluBwdRing = TileRing<3, kGluBwdSlots>;
struct GluBwdSmem {
  static constexpr int kEmit = (GluBwdRing::kBytes + 127) / 128 * 128;
  static constexpr int kAlloc = kEmit + TileEmit<2, false>::kBytes + 128;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 1)
    swiglu_bwd_tile_kernel(const __grid_constant__ CUtensorMap map_g,
                           const __grid_constant__ CUtensorMap map_u,
                           const __grid_constant__ CUtensorMap map_da, const GluTileArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const int count = tiles_of_block(a.tiles_r * a.tiles_c);
  GluBwdRing ring(smem, count);
  if (threadIdx.x == 0) {
    ring.init();
    prefetch_tmap(&map_g);
    prefetch_tmap(&map_u);
    prefetch_tmap(&map_da);
  }
  TileEmit<2, POW2>::init(smem + GluBwdSmem::kEmit);
  __syncthreads();
  launch_dependents();
  grid_dependency_wait();
  auto load = [&](int i, int n, uint32_t dst, uint32_t bar) {
    const int tile = static_cast<int>(blockIdx.x + i * gridDim.x);
    tma_load_2d(dst, n == 0 ? &map_g : n == 1 ? &map_u : &map_da, bar, (tile % a.tiles_c) * kTile,
                (tile / a.tiles_c) * kTile);
  };
  if (threadIdx.x == 0) ring.fill(kGluBwdSlots, load);
  TileEmit<2, POW2> emit(smem + GluBwdSmem::kEmit, a.out);
  for (int i = 0; i < count; ++i) {
    const int tile = static_cast<int>(blockIdx.x + i * gridDim.x);
    const int tr = tile / a.tiles_c, tc = tile % a.tiles_c;
    float y[2][8][4];
    const uint8_t* gate = ring.next();
    const uint8_t* up = ring.next();
    const uint8_t* da = ring.next();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float g[4], u[4], d[4];
      read4(gate, p, g);
      read4(up, p, u);
      read4(da, p, d);
#pragma unroll
      for (int j = 0; j < 4; j += 2) glu_grad2(g + j, u + j, d + j, &y[0][p][j], &y[1][p][j]);
    }
    emit.step(y, tr, {tc, tc + a.tiles_c}, [&] {
      if (threadIdx.x == 0) ring.fill(3, load);
    });
  }
  emit.finish();
  if (threadIdx.x == 0) ring.drain();
}

// Backward for f = 128 m + r, r > 0: the dup half of d then starts in the middle
// of a tile, so input tile s (columns 128 s ..) gives dgate's tile s, but dup
// values for two tiles of d: its first 128 - r columns end tile m + s, its last r
// begin tile m + s + 1. The lanes' columns of the dup tile are their input columns
// turned by r; one of the two parts waits in shared memory (fp32, for the thread
// that wrote it) for the block's next step, whose other part completes it. A block
// takes consecutive tiles of a row of tiles, upwards for r <= 64 (the last r
// columns are kept) and downwards beyond (the first 128 - r), so that half a tile
// is enough. Two pieces come from plain loads: what the block's first step would
// have been left by the one before it, and in tile m the first dup columns, which
// share it with the end of dgate.
// (16384 x 6128: 216 us. When it was 209: 214 with one run per block, for then the blocks are all
// over the tensor; 217 with the values shuffled into place instead of other columns
// per lane; 217 with the pieces of a run's start copied ahead, for the registers;
// 338 with the kernel below.)
constexpr int kGluShiftSlots = 5;
constexpr int kGluRun = 16;
using GluShiftRing = TileRing<3, kGluShiftSlots>;
struct GluShiftSmem {
  static constexpr int kEmit = (GluShiftRing::kBytes + 127) / 128 * 128;
  static constexpr int kKept = kEmit + TileEmit<2, false>::kBytes;   // half a tile
  static constexpr int kAlloc = kKept + kTile * kTile * 2 + 128;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};
struct GluShiftArgs {
  const uint16_t* gu;
  const uint16_t* da;
  int64_t rows;
  int f, tiles_r;
  CodesOut out;
};

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 1)
    swiglu_bwd_shift_kernel(const __grid_constant__ CUtensorMap map_g,
                            const __grid_constant__ CUtensorMap map_u,
                            const __grid_constant__ CUtensorMap map_da, const GluShiftArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const int m = a.f / kTile, r = a.f % kTile, per_row = m + 1;
  const bool down = r > kTile / 2;
  const int64_t total = static_cast<int64_t>(a.tiles_r) * per_row;
  // tiles in runs of kGluRun by all blocks in turn; what is left, in shorter ones
  const int full = static_cast<int>(total / (kGluRun * gridDim.x));
  const int64_t done = static_cast<int64_t>(full) * kGluRun * gridDim.x;
  const int last = static_cast<int>(done + (total - done) * blockIdx.x / gridDim.x);
  const int count =
      full * kGluRun + static_cast<int>(done + (total - done) * (blockIdx.x + 1) / gridDim.x) - last;
  auto tile_at = [&](int i) {
    const int k = i / kGluRun;
    return k < full ? static_cast<int>(k * gridDim.x + blockIdx.x) * kGluRun + i % kGluRun
                    : last + i - full * kGluRun;
  };
  GluShiftRing ring(smem, count);
  if (threadIdx.x == 0) {
    ring.init();
    prefetch_tmap(&map_g);
    prefetch_tmap(&map_u);
    prefetch_tmap(&map_da);
  }
  TileEmit<2, POW2>::init(smem + GluShiftSmem::kEmit);
  __syncthreads();
  launch_dependents();
  grid_dependency_wait();
  auto input_tile = [&](int t) { return down ? m - t % per_row : t % per_row; };
  auto load = [&](int i, int n, uint32_t dst, uint32_t bar) {
    const int t = tile_at(i);
    tma_load_2d(dst, n == 0 ? &map_g : n == 1 ? &map_u : &map_da, bar, input_tile(t) * kTile,
                t / per_row * kTile);
  };
  if (threadIdx.x == 0) ring.fill(kGluShiftSlots, load);
  TileEmit<2, POW2, true> emit(smem + GluShiftSmem::kEmit, a.out);

  const int rb = threadIdx.x >> 5, lane = threadIdx.x & 31, rot = r / 4;
  emit.turn = rot;
  const int dl = emit.lane_of(1);          // columns 4 dl .. of the dup tile
  const bool keeps = down ? dl >= rot : dl < rot;
  float4* kept = reinterpret_cast<float4*>(smem + GluShiftSmem::kKept) + rb * 8 * 16 +
                 (down ? dl - rot : dl);                       // of row p: at 16 p
  // dup of this thread's 8 rows of row tile tr, four columns from c on (0 outside):
  // all loads first, then `put(p, values)`
  auto dup_at = [&](int tr, int c, auto&& put) {
    const int64_t row = static_cast<int64_t>(tr) * kTile + rb * 8;
    uint2 wg[8], wd[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const bool in = row + p < a.rows && c >= 0 && c < a.f;
      wg[p] = wd[p] = make_uint2(0u, 0u);
      if (in) wg[p] = *reinterpret_cast<const uint2*>(a.gu + (row + p) * 2 * a.f + c);
      if (in) wd[p] = *reinterpret_cast<const uint2*>(a.da + (row + p) * a.f + c);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float g[4] = {bf16_lo(wg[p].x), bf16_hi(wg[p].x), bf16_lo(wg[p].y), bf16_hi(wg[p].y)};
      const float d[4] = {bf16_lo(wd[p].x), bf16_hi(wd[p].x), bf16_lo(wd[p].y), bf16_hi(wd[p].y)};
      float v[4], unused[2];
      glu_grad2(g, g, d, unused, v);
      glu_grad2(g + 2, g + 2, d + 2, unused, v + 2);
      put(p, v);
    }
  };
  for (int i = 0; i < count; ++i) {
    const int t = tile_at(i), tr = t / per_row, s = input_tile(t);
    if (i % kGluRun == 0 && keeps) {       // a run starts
      dup_at(tr, (down ? s + 1 : s) * kTile - r + dl * 4, [&](int p, const float(&v)[4]) {
        kept[16 * p] = make_float4(v[0], v[1], v[2], v[3]);
      });
    }
    float y[2][8][4];
    const uint8_t* gate = ring.next();
    const uint8_t* up = ring.next();
    const uint8_t* da = ring.next();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float g[4], u[4], d[4];
      read4(gate, p, g);
      read4(up, p, u);
      read4(da, p, d);
#pragma unroll
      for (int j = 0; j < 4; j += 2) glu_grad2(g + j, u + j, d + j, &y[0][p][j], &y[1][p][j]);
      if (keeps) {
        // (nothing lies right of tile m)
        const float4 k = down && s == m ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : kept[16 * p];
        kept[16 * p] = make_float4(y[1][p][0], y[1][p][1], y[1][p][2], y[1][p][3]);
        y[1][p][0] = k.x, y[1][p][1] = k.y, y[1][p][2] = k.z, y[1][p][3] = k.w;
      }
    }
    if (s == m && lane >= rot) {
      dup_at(tr, lane * 4 - r, [&](int p, const float(&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[0][p][j] = v[j];
      });
    }
    // upwards, the first step of a row only leaves its end behind: its other dup
    // columns are those of tile m (a tile past the end is not written)
    const int t1 = down ? m + s + 1 : s > 0 ? m + s : 2 * m + 2;
    emit.step(y, tr, {s, t1}, [&] {
      if (threadIdx.x == 0) ring.fill(3, load);
    });
  }
  emit.finish();
  if (threadIdx.x == 0) ring.drain();
}

// The same for no more tiles of d than two blocks per SM hold: each tile by itself,
// every 4-column run from its own gate, up and da columns (read twice in all, with
// plain loads). Half the work per block, and no second tile to wait for: 777 x 1360
// 7.0 us against 8.7 above, 1000 x 1360 7.8 and 9.2.
struct GluRaggedArgs {
  const uint16_t* gu;
  const uint16_t* da;
  int64_t rows, f;
  GluTileArgs t;            // tiles of the output's [rows, 2f]
};

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 2)
    swiglu_bwd_ragged_kernel(const GluRaggedArgs r) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const GluTileArgs& a = r.t;
  const int rb = threadIdx.x >> 5, lane = threadIdx.x & 31;
  TileEmit<1, POW2>::init(smem);
  __syncthreads();
  launch_dependents();
  grid_dependency_wait();
  TileEmit<1, POW2> emit(smem, a.out);
  const int tile = static_cast<int>(blockIdx.x);
  const int tr = tile / a.tiles_c, tc = tile % a.tiles_c;
  const int64_t c0 = static_cast<int64_t>(tc) * kTile + lane * 4;
  const bool is_up = c0 >= r.f;
  const int64_t src = is_up ? c0 - r.f : c0;
  float y[1][8][4];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t row = static_cast<int64_t>(tr) * kTile + rb * 8 + p;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[0][p][j] = 0.0f;
    if (row < r.rows && c0 < 2 * r.f) {
      const uint16_t* gp = r.gu + row * 2 * r.f + src;
      const uint2 wg = *reinterpret_cast<const uint2*>(gp);
      const uint2 wu = *reinterpret_cast<const uint2*>(gp + r.f);
      const uint2 wd = *reinterpret_cast<const uint2*>(r.da + row * r.f + src);
      const float g[4] = {bf16_lo(wg.x), bf16_hi(wg.x), bf16_lo(wg.y), bf16_hi(wg.y)};
      const float u[4] = {bf16_lo(wu.x), bf16_hi(wu.x), bf16_lo(wu.y), bf16_hi(wu.y)};
      const float d[4] = {bf16_lo(wd.x), bf16_hi(wd.x), bf16_lo(wd.y), bf16_hi(wd.y)};
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        float dgate[2], dup[2];
        glu_grad2(g + j, u + j, d + j, dgate, dup);
        y[0][p][j] = is_up ? dup[0] : dgate[0];
        y[0][p][j + 1] = is_up ? dup[1] : dgate[1];
      }
    }
  }
  emit.step(y, tr, {tc}, [] {});
  emit.finish();
}

}  // namespace layer
}  // namespace fp8bw
