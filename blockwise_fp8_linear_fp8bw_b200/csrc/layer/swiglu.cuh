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

// 1 / (1 + exp(-x)) by the fast exponential and division: relative error about
// (2 + |x|) * 2^-23. Below -87 the quotient is 0 (its value there is under
// 2^-125); at -inf it is 0, so that x * sigmoid(x) is NaN as the formula says.
__device__ __forceinline__ float sigmoid(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

// ---------------------------------------------------------------- row-wise only
struct GluRowArgs {
  const uint16_t* gu;
  int64_t rows, rows_pad, f;
  uint8_t* q;
  float* s;
};

constexpr int kGluRowThreads = 256;

// One half-warp per row and group; a block takes 16 rows of one group, so its
// scales are one 64-byte run.
template <bool POW2>
__global__ void __launch_bounds__(kGluRowThreads) swiglu_row_kernel(const GluRowArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 128 + (threadIdx.x & 15) * 8;
  const bool in = row < a.rows && c < a.f;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = 0.0f;
  if (in) {
    const uint16_t* p = a.gu + row * 2 * a.f + c;
    const uint4 wg = ld16_stream(p), wu = ld16_stream(p + a.f);
    float g[8], u[8];
    unpack8(wg, g);
    unpack8(wu, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = g[j] * sigmoid(g[j]) * u[j];
  }
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float qs, s;
  scale_of<POW2>(m, qs, s);
  if (row < a.rows_pad && c < a.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= qs;
    *reinterpret_cast<uint2*>(a.q + row * a.f + c) = encode8(y);
    if ((threadIdx.x & 15) == 0) a.s[static_cast<int64_t>(blockIdx.y) * a.rows_pad + row] = s;
  }
}

// ---------------------------------------------------------------- 128x128 tiles
struct GluTileArgs {
  int64_t rows_pad, f;
  int tiles_r, tiles_c;     // of [rows_pad, f]
  uint8_t* q;
  float* s;
  uint8_t* q_t;
  float* s_t;
};

// Forward: the gate and up tiles arrive by TMA in one buffer, which is
// refilled as soon as the products are in registers; two CTAs per SM keep
// loads in flight through each other's encoding.
struct GluFwdSmem {
  static constexpr int kIn = 0;                       // gate, up
  static constexpr int kEmit = 2 * kTileBytes;
  static constexpr int kBar = kEmit + TileEmit::kBytes;
  static constexpr int kBytes = kBar + 32;
  static constexpr int kAlloc = kBytes + 128;
};

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 2)
    swiglu_tile_kernel(const __grid_constant__ CUtensorMap map_g,
                       const __grid_constant__ CUtensorMap map_u, const GluTileArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar = sbase + GluFwdSmem::kBar;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + GluFwdSmem::kBar + 16);
  const int t = threadIdx.x, rb = t >> 4, cg = t & 15;
  const int num_tiles = a.tiles_r * a.tiles_c;
  if (t == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    prefetch_tmap(&map_g);
    prefetch_tmap(&map_u);
  }
  __syncthreads();
  launch_dependents();
  grid_dependency_wait();
  auto load = [&](int tile) {
    const int x = (tile % a.tiles_c) * kTile, y = (tile / a.tiles_c) * kTile;
    mbar_arrive_expect_tx(bar, 2 * kTileBytes);
    tma_load_2d(sbase + GluFwdSmem::kIn, &map_g, bar, x, y);
    tma_load_2d(sbase + GluFwdSmem::kIn + kTileBytes, &map_u, bar, x, y);
  };
  int pend[1] = {-1};
  if (t == 0 && blockIdx.x < num_tiles) {
    load(blockIdx.x);
    pend[0] = 0;
  }
  int i = 0;
  for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++i) {
    const bool got = mbar_wait(bar, i & 1, abort_flag, kErrTimeoutTma);
    if (!__syncthreads_and(got ? 1 : 0)) break;
    pend[0] = -1;
    float y[8][8];
    const uint16_t* in = reinterpret_cast<const uint16_t*>(smem + GluFwdSmem::kIn);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int at = (rb * 8 + p) * kTile + cg * 8;
      float g[8], u[8];
      unpack8(ld16(in + at), g);
      unpack8(ld16(in + kTile * kTile + at), u);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[p][j] = g[j] * sigmoid(g[j]) * u[j];
    }
    __syncthreads();   // the buffer is free
    if (t == 0 && tile + gridDim.x < num_tiles) {
      load(tile + gridDim.x);
      pend[0] = (i + 1) & 1;
    }
    const TileOut o{a.q, a.s, a.q_t, a.s_t, a.rows_pad, a.f, tile / a.tiles_c, tile % a.tiles_c};
    emit_tile<true, true, POW2>(y, smem + GluFwdSmem::kEmit, o);
  }
  if (t == 0) drain_loads(bar, pend, 1);
}

// Backward, f a multiple of 128 (so that the groups of d do not straddle its
// two halves): gate, up and da tiles in; two output tiles (dgate, dup). Each
// thread computes both gradients of its 8x8 sub-block at once and parks dup,
// in fp32, in the shared memory its own gate and up values came from (the same
// 256 bytes), so exp is evaluated once and registers hold one tile.
struct GluBwdSmem {
  static constexpr int kIn = 0;                       // gate, up, da
  static constexpr int kEmit = 3 * kTileBytes - 16 * 1024;  // T overlays da's second half
  static constexpr int kBar = kEmit + TileEmit::kBytes;
  static constexpr int kBytes = kBar + 32;
  static constexpr int kAlloc = kBytes + 128;
};
static_assert(TileEmit::kT == 0 && kTile * kTile == 16 * 1024, "T overlays half of the da tile");

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 2)
    swiglu_bwd_tile_kernel(const __grid_constant__ CUtensorMap map_g,
                           const __grid_constant__ CUtensorMap map_u,
                           const __grid_constant__ CUtensorMap map_da, const GluTileArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar = sbase + GluBwdSmem::kBar;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + GluBwdSmem::kBar + 16);
  const int t = threadIdx.x, rb = t >> 4, cg = t & 15;
  const int num_tiles = a.tiles_r * a.tiles_c;
  if (t == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    prefetch_tmap(&map_g);
    prefetch_tmap(&map_u);
    prefetch_tmap(&map_da);
  }
  __syncthreads();
  launch_dependents();
  grid_dependency_wait();
  int i = 0;
  for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++i) {
    const int tr = tile / a.tiles_c, tc = tile % a.tiles_c;
    if (t == 0) {
      mbar_arrive_expect_tx(bar, 3 * kTileBytes);
      tma_load_2d(sbase, &map_g, bar, tc * kTile, tr * kTile);
      tma_load_2d(sbase + kTileBytes, &map_u, bar, tc * kTile, tr * kTile);
      tma_load_2d(sbase + 2 * kTileBytes, &map_da, bar, tc * kTile, tr * kTile);
    }
    const bool got = mbar_wait(bar, i & 1, abort_flag, kErrTimeoutTma);
    if (!__syncthreads_and(got ? 1 : 0)) {
      if (t == 0) {
        const int pend[1] = {i & 1};
        drain_loads(bar, pend, 1);
      }
      break;
    }
    float y[8][8];
    uint8_t* in = smem;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int at = ((rb * 8 + p) * kTile + cg * 8) * 2;
      float g[8], u[8], d[8];
      unpack8(ld16(in + at), g);
      unpack8(ld16(in + kTileBytes + at), u);
      unpack8(ld16(in + 2 * kTileBytes + at), d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sg = sigmoid(g[j]);
        const float w = d[j] * sg;
        y[p][j] = w * u[j] * fmaf(g[j], 1.0f - sg, 1.0f);
        u[j] = w * g[j];
      }
      *reinterpret_cast<float4*>(in + at) = make_float4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<float4*>(in + kTileBytes + at) = make_float4(u[4], u[5], u[6], u[7]);
    }
    __syncthreads();   // da's buffer is free: it holds the transposed codes now
    TileOut o{a.q, a.s, a.q_t, a.s_t, a.rows_pad, 2 * a.f, tr, tc};
    emit_tile<true, true, POW2>(y, smem + GluBwdSmem::kEmit, o);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int at = ((rb * 8 + p) * kTile + cg * 8) * 2;
      const float4 lo = *reinterpret_cast<const float4*>(in + at);
      const float4 hi = *reinterpret_cast<const float4*>(in + kTileBytes + at);
      y[p][0] = lo.x, y[p][1] = lo.y, y[p][2] = lo.z, y[p][3] = lo.w;
      y[p][4] = hi.x, y[p][5] = hi.y, y[p][6] = hi.z, y[p][7] = hi.w;
    }
    o.tc = tc + a.tiles_c;
    emit_tile<true, true, POW2, true>(y, smem + GluBwdSmem::kEmit, o);
  }
}

// Backward for f no multiple of 128: the 1x128 groups of d then straddle the
// dgate/dup boundary, so each tile of d's 2f columns is computed by itself,
// every 8-column run from its own gate, up and da columns (read twice in all,
// with plain loads).
struct GluRaggedArgs {
  const uint16_t* gu;
  const uint16_t* da;
  int64_t rows;
  GluTileArgs t;            // tiles of [rows_pad, 2f]
};

template <bool POW2>
__global__ void __launch_bounds__(kTileThreads, 2)
    swiglu_bwd_ragged_kernel(const GluRaggedArgs r) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const GluTileArgs& a = r.t;
  const int t = threadIdx.x, rb = t >> 4, cg = t & 15;
  const int num_tiles = a.tiles_r * a.tiles_c;
  launch_dependents();
  grid_dependency_wait();
  for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
    const int tr = tile / a.tiles_c, tc = tile % a.tiles_c;
    const int64_t c0 = static_cast<int64_t>(tc) * kTile + cg * 8;
    const bool is_up = c0 >= a.f;
    const int64_t src = is_up ? c0 - a.f : c0;
    float y[8][8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int64_t row = static_cast<int64_t>(tr) * kTile + rb * 8 + p;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[p][j] = 0.0f;
      if (row < r.rows && c0 < 2 * a.f) {
        const uint16_t* gp = r.gu + row * 2 * a.f + src;
        float g[8], u[8], d[8];
        unpack8(ld16(gp), g);
        unpack8(ld16(gp + a.f), u);
        unpack8(ld16(r.da + row * a.f + src), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float sg = sigmoid(g[j]);
          const float w = d[j] * sg;
          y[p][j] = is_up ? w * g[j] : w * u[j] * fmaf(g[j], 1.0f - sg, 1.0f);
        }
      }
    }
    const TileOut o{a.q, a.s, a.q_t, a.s_t, a.rows_pad, 2 * a.f, tr, tc};
    emit_tile<true, true, POW2>(y, smem, o);
  }
}

}  // namespace layer
}  // namespace fp8bw
