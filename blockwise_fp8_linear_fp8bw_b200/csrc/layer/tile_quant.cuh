// tile_quant.cuh -- E4M3 quantisation of 128x128 tiles of fp32 values that a
// kernel holds in registers: row-wise codes with 1x128 scales and
// column-wise codes (transposed) with 128x1 scales, with the arithmetic and
// layouts of the quantisers.
//
// 512 threads: warp w owns rows 8w .. 8w+7 of the tile and lane l the columns
// 4l .. 4l+3, so a warp holds eight whole 1x128 groups and a thread 32 values per
// tile (two tiles at once fit its registers). A ring of input tiles is kept
// filled by TMA.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "../common.cuh"

namespace fp8bw {
namespace layer {

constexpr int kTile = 128;
constexpr int kTileThreads = 512;
constexpr int kTileBytes = kTile * kTile * 2;   // one bf16 tile

__device__ __forceinline__ uint8_t* align128(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 127) &
                                    ~static_cast<uintptr_t>(127));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// The block's tiles: blockIdx.x, blockIdx.x + gridDim.x, ...
__device__ __forceinline__ int tiles_of_block(int num_tiles) {
  return (num_tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
         static_cast<int>(gridDim.x);
}

// Four values as E4M3 (round to nearest even, saturating), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four values times k, as E4M3.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float k) {
  fmul2(a, b, a, b, k, k);
  fmul2(c, d, c, d, k, k);
  return e4m3x4(a, b, c, d);
}

// max(m, |a|, |b|) in one instruction.
__device__ __forceinline__ float max3_abs(float m, float a, float b) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

// 448 / amax: the approximate reciprocal (of amax / 16, so that no finite amax has a
// subnormal one) and a correction by what the product leaves of 448. It equals the
// correctly rounded quotient for every positive fp32 amax (compared with IEEE
// division over all of them), as near_over_448 does where 448 / amax is finite.
// 0 for infinity, infinite or NaN where the quotient is.
__device__ __forceinline__ float near_448_over(float amax) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(amax * 0.0625f));
  const float q = 28.0f * r, e = fmaf(-q, amax, 448.0f);
  return fabsf(e) < 1.0f ? fmaf(e * 0.0625f, r, q) : q;
}

// amax / 448, corrected in the same way.
__device__ __forceinline__ float near_over_448(float amax) {
  const float q = amax * (1.0f / 448.0f);
  return isfinite(amax) ? fmaf(fmaf(-q, 448.0f, amax), 1.0f / 448.0f, q) : q;
}

// scale_of for the fused kernels: the same scales without IEEE divisions (some 40
// instructions and their latency, in every step).
template <bool POW2>
__device__ __forceinline__ void scale_near(float amax, float& qscale, float& s) {
  if constexpr (POW2) {
    group_scale_pow2(amax, qscale, s);
  } else {
    const float r = near_448_over(amax);
    const bool none = !isfinite(r) || amax == 0.0f;
    qscale = none ? 1.0f : r;
    s = none ? 1.0f : near_over_448(amax);
  }
}

// Largest |v| of the warp, in every lane.
__device__ __forceinline__ float warp_max_abs(float v) {
  float r;
  asm volatile("redux.sync.max.abs.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}

// Where codes and scales go (the column-wise ones may be unused).
struct CodesOut {
  uint8_t* q;          // [rows][cols]
  float* s;            // [ceil(cols/128)][rows]
  uint8_t* q_t;        // [cols][rows]
  float* s_t;          // [ceil(rows/128)][cols]
  int64_t rows, cols;  // rows padded to a multiple of 16; cols is one too
};

// Byte offset in a transposed tile of the 8-byte unit of tokens 8u .. 8u+7 of
// column k. Units are xor-ed with the 4-column block (the 32 columns that a
// warp writes at once, 4 apart, land in all 16 bank pairs) and with the column's
// parity (the four columns that it reads at once use even and odd units).
__device__ __forceinline__ int emit_t_offset(int k, int u) {
  return k * kTile + ((u ^ (k >> 2) ^ (k & 1)) & 15) * 8;
}

// Writes the codes of NOUT tiles per step, all of row tile tr, from the 8x4
// values of each thread; entries outside the tensor must be zero (a whole tile
// may lie outside). Column
// scales need the whole tile, so a step has two barriers. To have work between
// them, the transposed codes of a step leave shared memory during the next one:
// between the barriers lie this step's row codes, the last step's transposed
// codes and (in a few warps) the column scales.
// With TURN, lane l holds columns 4 l' .. of the second tile, l' = (l + turn) % 32.
template <int NOUT, bool POW2, bool TURN = false>
struct TileEmit {
  static constexpr int kT = 0;                                   // NOUT x 16 KB
  // Column maxima, combined by shared-memory atomics on the bits (they are not
  // negative, and a maximum does not depend on the order). One slot per warp and
  // column would take 8 KB a tile, which the input ring needs more: the gated
  // product's backward pass took 230, 199 and 181 us with 3, 4 and 5 ring tiles, and
  // 167 with the 6 that fit (170 with the present scales).
  static constexpr int kRed = kT + NOUT * kTile * kTile;         // NOUT x 128
  static constexpr int kColQ = kRed + NOUT * kTile * 4;          // NOUT x 128 floats
  static constexpr int kBytes = kColQ + NOUT * kTile * 4;

  uint8_t* smem;
  const CodesOut& out;
  int64_t row_at, col_at;      // offsets in a tile of q (its rows) and of q_t
  int last_tr = -1, last_tc[NOUT];
  int turn = 0;

  __device__ __forceinline__ int lane_of(int n) const {
    const int lane = threadIdx.x & 31;
    return TURN && n == 1 ? (lane + turn) & 31 : lane;
  }

  // All threads, before the block's first barrier.
  __device__ __forceinline__ static void init(uint8_t* p) {
    if (threadIdx.x < NOUT * kTile) reinterpret_cast<int*>(p + kRed)[threadIdx.x] = 0;
  }

  __device__ __forceinline__ TileEmit(uint8_t* p, const CodesOut& o) : smem(p), out(o) {
    const int t = threadIdx.x;
    row_at = static_cast<int64_t>((t >> 5) * 8) * o.cols;
    col_at = static_cast<int64_t>(t >> 3) * o.rows + (t & 7) * 16;
  }

  // What is left of the tensor from tile index i on (sizes fit 31 bits).
  __device__ __forceinline__ static int left(int64_t size, int i) {
    return static_cast<int>(size) - i * kTile;
  }

  // `freed()` runs after the first barrier: every thread is past reading the
  // inputs that y came from.
  template <typename Freed>
  __device__ __forceinline__ void step(const float (&y)[NOUT][8][4], int tr,
                                       const int (&tc)[NOUT], Freed&& freed) {
    const int t = threadIdx.x, rb = t >> 5;
    int* red = reinterpret_cast<int*>(smem + kRed);
    float* colq = reinterpret_cast<float*>(smem + kColQ);
    // column maxima of this warp's 8 rows
#pragma unroll
    for (int n = 0; n < NOUT; ++n) {
      float m[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = max3_abs(0.0f, y[n][0][j], y[n][1][j]);
#pragma unroll
        for (int p = 2; p < 8; p += 2) m[j] = max3_abs(m[j], y[n][p][j], y[n][p + 1][j]);
      }
      // column 4l + j at 32j + l: a warp's 32 addresses are in 32 banks
#pragma unroll
      for (int j = 0; j < 4; ++j)
        atomicMax(red + n * kTile + j * 32 + lane_of(n), __float_as_int(m[j]));
    }
    __syncthreads();
    freed();
    if (t < NOUT * kTile) {
      const int n = t >> 7, k = t & 127;
      int* r = red + n * kTile + (k & 3) * 32 + (k >> 2);
      const float m = __int_as_float(*r);
      *r = 0;
      float qs, s;
      scale_near<POW2>(m, qs, s);
      colq[t] = qs;
      const int c = NOUT == 1 || n == 0 ? tc[0] : tc[NOUT - 1];
      if (k < left(out.cols, c))
        out.s_t[static_cast<int64_t>(tr) * out.cols + static_cast<int64_t>(c) * kTile + k] = s;
    }
    if (last_tr >= 0) write_transposed();
#pragma unroll
    for (int n = 0; n < NOUT; ++n) write_rows(y[n], tr, tc[n], lane_of(n));
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NOUT; ++n) {
      uint8_t* T = smem + kT + n * kTile * kTile;
      const int lane = lane_of(n);
      const float4 k4 = *reinterpret_cast<const float4*>(colq + n * kTile + lane * 4);
      float v[8][4];
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        fmul2(v[p][0], v[p][1], y[n][p][0], y[n][p][1], k4.x, k4.y);
        fmul2(v[p][2], v[p][3], y[n][p][2], y[n][p][3], k4.z, k4.w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2*>(T + emit_t_offset(lane * 4 + j, rb)) =
            make_uint2(e4m3x4(v[0][j], v[1][j], v[2][j], v[3][j]),
                       e4m3x4(v[4][j], v[5][j], v[6][j], v[7][j]));
      last_tc[n] = tc[n];
    }
    last_tr = tr;
  }

  // After the last step.
  __device__ __forceinline__ void finish() {
    if (last_tr < 0) return;
    __syncthreads();
    write_transposed();
  }

  __device__ __forceinline__ void write_transposed() const {
    const int kk = threadIdx.x >> 3, ch = threadIdx.x & 7;
    const bool rin = ch * 16 < left(out.rows, last_tr);
#pragma unroll
    for (int n = 0; n < NOUT; ++n) {
      // tile column k is 128 contiguous tokens of row tc*128 + k of q_t
      const uint8_t* T = smem + kT + n * kTile * kTile;
      const int cols = left(out.cols, last_tc[n]);
      uint8_t* dst = out.q_t + static_cast<int64_t>(last_tc[n]) * kTile * out.rows +
                     static_cast<int64_t>(last_tr) * kTile + col_at;
#pragma unroll
      for (int k0 = 0; k0 < kTile; k0 += kTileThreads / 8) {
        const uint2 lo = *reinterpret_cast<const uint2*>(T + emit_t_offset(k0 + kk, 2 * ch));
        const uint2 hi = *reinterpret_cast<const uint2*>(T + emit_t_offset(k0 + kk, 2 * ch + 1));
        if (rin && k0 + kk < cols)
          *reinterpret_cast<uint4*>(dst + k0 * out.rows) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }

  // `col`: the lane whose columns this one holds
  __device__ __forceinline__ void write_rows(const float (&y)[8][4], int tr, int tc,
                                             int col) const {
    const int rb = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // row maxima; lane l computes the scale of row l & 7
    float mine = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float m = warp_max_abs(max3_abs(max3_abs(0.0f, y[p][0], y[p][1]), y[p][2], y[p][3]));
      if ((lane & 7) == p) mine = m;
    }
    float qs, s;
    scale_near<POW2>(mine, qs, s);
    // rows is a multiple of 16: the warp's 8 rows are all in or all out
    const bool rin = rb * 8 < left(out.rows, tr) && left(out.cols, tc) > 0;
    const int64_t r0 = static_cast<int64_t>(tr) * kTile;
    if (lane < 8 && rin) out.s[static_cast<int64_t>(tc) * out.rows + r0 + rb * 8 + lane] = s;
    uint8_t* q = out.q + r0 * out.cols + static_cast<int64_t>(tc) * kTile + row_at + col * 4;
    const bool in = rin && col * 4 < left(out.cols, tc);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float k = __shfl_sync(0xFFFFFFFFu, qs, p);
      const uint32_t code = encode4(y[p][0], y[p][1], y[p][2], y[p][3], k);
      if (in) *reinterpret_cast<uint32_t*>(q) = code;
      q += out.cols;
    }
  }
};

// ---------------------------------------------------------------- columns alone
// Column-wise codes of a 128 x 64 tile by 256 threads: thread t holds rows
// 8 * (t / 16) .. +7 and columns 4 * (t % 16) .. +3.
constexpr int kColTile = 64;
constexpr int kColThreads = 256;

struct ColumnsSmem {
  float red[kColThreads / 32][kColTile];
  float q[kColTile];
  float q2[kColTile];
  __align__(16) uint8_t t[kColTile * kTile];
};

// Gain of a product that has none.
struct NoGain {
  __device__ __forceinline__ float operator()(int64_t) const { return 1.0f; }
};

// Of y times gain(column), from the thread's column maxima m of |y|; entries outside
// the tensor must be zero, and are in the codes whatever the gain: `live` of the
// thread's rows are inside.
template <bool POW2, typename Gain>
__device__ __forceinline__ void emit_columns(ColumnsSmem& sm, float (&y)[8][4], float (&m)[4],
                                             int tr, int tc, int64_t rows_pad, int64_t cols,
                                             uint8_t* q_t, float* s_t, int live, Gain&& gain) {
  constexpr bool kGain = !std::is_same<std::decay_t<Gain>, NoGain>::value;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, rb = t >> 4, cb = t & 15;
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
  if (lane < 16)
    *reinterpret_cast<float4*>(&sm.red[warp][cb * 4]) = make_float4(m[0], m[1], m[2], m[3]);
  __syncthreads();
  bool odd = false;
  if (t < kColTile) {
    const int64_t c = static_cast<int64_t>(tc) * kColTile + t;
    float am = sm.red[0][t];
#pragma unroll
    for (int i = 1; i < kColThreads / 32; ++i) am = fmaxf(am, sm.red[i][t]);
    float qs, s;
    if constexpr (kGain) {
      const float g = c < cols ? gain(c) : 0.0f;
      const float top = am * fabsf(g);
      scale_near<POW2>(top, qs, s);
      float k = qs * g;
      if constexpr (!POW2) {
        // the gain cancels: +-448 / max|y| (not where a scale of 1 stands for none, or
        // something is not finite)
        const float d = near_448_over(am);
        if (isfinite(d) && qs > 0.0f && !(qs == 1.0f && s == 1.0f)) k = copysignf(d, g);
      }
      // where one factor for gain and scale may leave fp32's range: one after the other
      odd = !(am >= 0x1p-100f && top <= 0x1p120f) && am != 0.0f;
      sm.q[t] = odd ? g : k;
      sm.q2[t] = odd ? qs : 1.0f;
    } else {
      scale_near<POW2>(am, qs, s);
      sm.q[t] = qs;
    }
    if (c < cols) s_t[static_cast<int64_t>(tr) * cols + c] = s;
  }
  bool twice = false;
  if constexpr (kGain) twice = __syncthreads_or(odd) != 0;
  else __syncthreads();
  const float4 k = *reinterpret_cast<const float4*>(&sm.q[cb * 4]);
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    fmul2(y[p][0], y[p][1], y[p][0], y[p][1], k.x, k.y);
    fmul2(y[p][2], y[p][3], y[p][2], y[p][3], k.z, k.w);
  }
  if constexpr (kGain) {
    if (twice) {
      const float4 k2 = *reinterpret_cast<const float4*>(&sm.q2[cb * 4]);
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        fmul2(y[p][0], y[p][1], y[p][0], y[p][1], k2.x, k2.y);
        fmul2(y[p][2], y[p][3], y[p][2], y[p][3], k2.z, k2.w);
      }
    }
    if (live < 8) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        if (p < live) continue;
        y[p][0] = y[p][1] = y[p][2] = y[p][3] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint2*>(sm.t + emit_t_offset(cb * 4 + j, rb)) =
        make_uint2(e4m3x4(y[0][j], y[1][j], y[2][j], y[3][j]),
                   e4m3x4(y[4][j], y[5][j], y[6][j], y[7][j]));
  __syncthreads();
  // tile column kk is 128 contiguous tokens of row tc*64 + kk of q_t
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int kk = i * 32 + (t >> 3), ch = t & 7;
    const int64_t c = static_cast<int64_t>(tc) * kColTile + kk;
    const int64_t tok = static_cast<int64_t>(tr) * kTile + ch * 16;
    const uint2 lo = *reinterpret_cast<const uint2*>(sm.t + emit_t_offset(kk, 2 * ch));
    const uint2 hi = *reinterpret_cast<const uint2*>(sm.t + emit_t_offset(kk, 2 * ch + 1));
    if (c < cols && tok < rows_pad)
      *reinterpret_cast<uint4*>(q_t + c * rows_pad + tok) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

// ---------------------------------------------------------------- input ring
// A ring of SLOTS bf16 tiles, filled by thread 0 and read by all; the i-th step
// of a block takes the NIN tiles i*NIN .. i*NIN+NIN-1 of its sequence. Every wait
// is bounded. After an expired one the threads go on through their remaining
// steps (the abort flag ends every further wait), so that all of them meet at
// every barrier.
template <int NIN, int SLOTS>
struct TileRing {
  static_assert(SLOTS >= NIN, "a step's inputs fit the ring");
  static constexpr int kBar = SLOTS * kTileBytes;
  static constexpr int kBytes = kBar + SLOTS * 8 + 16;

  uint8_t* base;
  uint32_t bar;
  volatile uint32_t* abort;
  int slot = 0;              // next to read ...
  uint32_t phase = 0;
  int fill_slot = 0, filled = 0, total;      // ... and to fill (thread 0)

  __device__ __forceinline__ TileRing(uint8_t* p, int steps)
      : base(p), bar(smem_u32(p) + kBar),
        abort(reinterpret_cast<volatile uint32_t*>(p + kBar + SLOTS * 8)), total(steps * NIN) {}
  __device__ __forceinline__ void init() const {      // one thread
    for (int s = 0; s < SLOTS; ++s) mbar_init(bar + 8u * s, 1);
    *abort = 0u;
    fence_mbar_init();
  }
  // Thread 0: load up to `count` tiles more; `load(i, n, dst, bar)` issues the
  // load of input n of step i. Their slots must be free.
  template <typename Load>
  __device__ __forceinline__ void fill(int count, Load&& load) {
    for (int k = 0; k < count && filled < total; ++k, ++filled) {
      const uint32_t b = bar + 8u * fill_slot;
      mbar_arrive_expect_tx(b, kTileBytes);
      load(filled / NIN, filled % NIN, smem_u32(base) + fill_slot * kTileBytes, b);
      if (++fill_slot == SLOTS) fill_slot = 0;
    }
  }
  // The next input, or nullptr after an expired wait.
  __device__ __forceinline__ const uint8_t* next() {
    const uint8_t* p = mbar_wait(bar + 8u * slot, phase, abort, kErrTimeoutTma)
                           ? base + slot * kTileBytes
                           : nullptr;
    if (++slot == SLOTS) {
      slot = 0;
      phase ^= 1u;
    }
    return p;
  }
  // Thread 0, after the last step: the block's shared memory must outlive the
  // copies into it, even if their readers gave up (every copy has then been
  // waited for already, and these return at once).
  __device__ __forceinline__ void drain() const {
    for (int k = filled > SLOTS ? filled - SLOTS : 0; k < filled; ++k) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar + 8u * (k % SLOTS), (k / SLOTS) & 1) &&
             globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
  }
};

// This thread's four values of row p of its 8x4 block (zeros without a tile).
__device__ __forceinline__ void read4(const uint8_t* tile, int p, float (&f)[4]) {
  if (tile == nullptr) {
    f[0] = f[1] = f[2] = f[3] = 0.0f;
    return;
  }
  const int rb = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint2 w = *reinterpret_cast<const uint2*>(tile + (rb * 8 + p) * (kTile * 2) + lane * 8);
  f[0] = bf16_lo(w.x);
  f[1] = bf16_hi(w.x);
  f[2] = bf16_lo(w.y);
  f[3] = bf16_hi(w.y);
}

}  // namespace layer
}  // namespace fp8bw
