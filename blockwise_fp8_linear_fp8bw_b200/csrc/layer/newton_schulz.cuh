// newton_schulz.cuh -- orthogonalisation of weight updates by Newton-Schulz
// products on the tensor cores (sm_100a, tcgen05 on CTA pairs).
//
//   X_0 = G / (||G||_F + eps)
//   A = X X^T,  P = a I + b A + c A A,  X <- P X          (rows <= columns)
//   A = X^T X,  P = a I + b A + c A A,  X <- X P          (rows >  columns)
// so A and P are r x r with r the shorter side (R the longer one). Every product
// is a launch of one GEMM kernel over all jobs (matrices) of the call; products
// of A, P and the like are symmetric: only tiles on and above the diagonal are
// computed, the others written as their mirror images from the same registers.
//
// A step on its own is three products (r^2 R, r^3 and 2 r^2 R flops). Two steps
// in a row can be taken on the short side alone, for A, P and their products
// commute:
//   A_1 = P_0 A_0 P_0,   X_2 = (P_1 P_0) X_0
// which saves the first of the two updates and the second Gram product (3 r^2 R)
// for three products more (T = P_0 A_0, A_1 = T P_0, P_1 P_0; r^3 each). That pays
// for oblong matrices. What is lost is that A_1 is no longer made from an X that
// exists: its rounding errors are amplified by up to a^2 = 12 for small singular
// values. That is harmless in the first pair (A is small) and in the last (no
// singular value is), so only those are taken so: for five steps 2 + 1 + 2. (And for
// matrices whose short side is one tile, where it saves launches: see the chain below.)
// (Simulated against 64 bits, 256 x 1536, errors of the bf16 result: Gaussian
// matrix 1.9e-3 step by step, 2.0e-3 with pairs; some directions 300 times the
// rest 1.8e-3 and 2.3e-3; all steps in one pair-like run: not finite.)
//
// Numbers. Operands are fp16 (11 significant bits; bf16's 8 lose 1% of the
// result in five steps), products accumulate in fp32. The iterate itself is
// held in 32 bits, as an fp16 pair x = hi + lo/2048 (22 significant bits): hi
// is the operand, and the pair is what a X is computed from. Rounding the
// iterate to hi alone would put noise of 2^-12 of the largest directions into
// all others, which the iteration then amplifies by a = 3.4 a step. fp16's
// range is kept by powers of two: X is stored times 2^10, A and B times 2^12.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "../common.cuh"

namespace fp8bw {
namespace ns {

constexpr int kMaxJobs = 8;
constexpr int BM = 128;            // rows per CTA; a pair computes 256
constexpr int BK = 128;            // contraction chunk: two blocks of 64 (128 bytes)
constexpr int kThreads = 384;
constexpr int kFirstEpiWarp = 4;
constexpr int kNumEpiWarps = 8;
constexpr float kXScale = 1024.0f;     // X is stored times this
constexpr float kAScale = 4096.0f;     // A, P - d I and T are stored times this
constexpr float kQScale = 1024.0f;     // P_1 P_0 - d_1 d_0 I is stored times this
constexpr float kLoScale = 2048.0f;    // lo = (x - hi) * this

constexpr int kShiftStep = 3;

// result = alpha * product + beta * C + beta2 * C2, minus diag on the diagonal
struct Job {
  int rows, cols;            // output; cols as stored (its pitch), including padding columns
  int tiles_n;               // tiles of BN columns per row of tiles
  int chunks;                // of the contraction
  int tile_end;              // cumulative tile count
  int pitch;                 // elements per row of C and C2
  uint8_t a_mn, b_mn;        // operand stored with the contraction outermost
  uint8_t sym;               // symmetric result: see above
  uint8_t split;             // the result is an iterate: hi to out, lo to lo
  uint8_t bf16;              // the result is bf16, not fp16
  const uint16_t* c;         // may be null
  const uint16_t* c2;        // may be null
  uint16_t* out;
  uint16_t* lo;              // of a split result; may be c2
  float alpha, beta, beta2, diag;
};

// Matrices in the workspace have rows of a multiple of 64 elements, the padding
// columns zero, so that a 3-D view [column block][row][64] is exact and one copy
// can bring two blocks: an operand's share of a chunk is one 32 KB box. (On one SM the
// TMA unit spends about 120 cycles on a box besides 64 bytes a cycle: boxes of 8, 16
// and 32 KB reach 64, 84 and 101 GB/s.)
struct Maps {
  CUtensorMap a[kMaxJobs];     // operands
  CUtensorMap b[kMaxJobs];
};

struct Args {
  Job job[kMaxJobs];
  int count;
};

template <int BN_>
struct Layout {
  static constexpr int BN = BN_;
  static constexpr int kStages = BN == 256 ? 3 : 4;
  static constexpr int kTmemBufs = 512 / BN;
  static constexpr int kABytes = BM * BK * 2;
  static constexpr int kBBytes = (BN / 2) * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kBoxBytes = 32 * 32 * 2;
  static constexpr int kSlotBytes = 2 * kBoxBytes;   // staging of a result box, per warp
  static constexpr int kSlotOff = kRingBytes;
  static constexpr int kBarOff = kSlotOff + kNumEpiWarps * kSlotBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kTmemBufs + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kBytes = kMiscOff + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

// A box of a 3-D tensor; as tma_load_2d_pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::"
      "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// kind::f16 instruction descriptor: fp32 accumulator, fp16 operands, majorness
// of A (bit 15) and B (bit 16), N >> 3 at bit 17, M >> 4 at bit 24.
__device__ __forceinline__ uint32_t idesc_f16(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// A box of 32 x 32 16-bit values staged in shared memory: rows of 64 bytes, the
// 16-byte units of row i exchanged by (i >> 1) & 3.
__device__ __forceinline__ uint32_t box_unit(uint32_t box, int row, int unit) {
  return box + row * 64 + ((unit ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void lds16(uint32_t at, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(at)
               : "memory");
}

// Units loaded eight rows at a time into a box.
__device__ __forceinline__ void put_rows(uint32_t box, const uint4 (&c)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    sts16(box_unit(box, 8 * i + (lane >> 2), lane & 3), c[i].x, c[i].y, c[i].z, c[i].w);
}

// A box to rows y.. and columns x.. of `out`, as far as they exist: eight rows of
// 64 bytes per instruction.
__device__ __forceinline__ void store_box(uint16_t* out, int rows, int cols, int y, int x,
                                          uint32_t box, int lane) {
  const int u = lane & 3;
  if (x + 8 * u >= cols) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rr = 8 * i + (lane >> 2);
    uint32_t w[4];
    lds16(box_unit(box, rr, u), w);
    if (y + rr < rows)
      *reinterpret_cast<uint4*>(out + static_cast<int64_t>(y + rr) * cols + x + 8 * u) =
          make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// v += k * (32 fp16 values).
__device__ __forceinline__ void add_scaled(float (&v)[32], const uint32_t (&w)[4][4], float k) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_f16(w[u][e]);
      ffma2(v[8 * u + 2 * e], v[8 * u + 2 * e + 1], f.x, f.y, k, k);
    }
  }
}

// The same of the lane's row of a box.
__device__ __forceinline__ void add_scaled(float (&v)[32], uint32_t box, float k, int lane) {
  uint32_t w[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) lds16(box_unit(box, lane, u), w[u]);
  add_scaled(v, w, k);
}

// Tile `lt` of a job -> (tm, tn). Symmetric results number only the tiles that
// reach the diagonal's 256-row block or lie right of it.
template <int BN>
__device__ __forceinline__ void tile_at(const Job& job, int lt, int& tm, int& tn) {
  if (job.sym) {
    constexpr int kPer = 256 / BN;
    tm = 0;
    int left = job.tiles_n;
    while (lt >= left) {
      lt -= left;
      left -= kPer;
      ++tm;
    }
    tn = tm * kPer + lt;
  } else {
    tm = lt / job.tiles_n;
    tn = lt - tm * job.tiles_n;
  }
}

// Output tiles of 256 x BN by clusters of two CTAs, each CTA holding 128 rows
// of A and BN/2 rows of B per chunk; roles as in the blockwise GEMMs: warp 0
// loads operands, warp 1 of the even CTA issues the MMAs, warps 4-11 read TMEM
// and write the result box by box (32 x 32). C and the result pass through shared
// memory, so that rows of 64 bytes are read and written eight at a time (lanes
// reading C row by row: 1.5% slower). The
// product of a whole tile stays in TMEM (512 / BN tiles fit), so the epilogue
// of one tile runs under the MMAs of the next. Eight 2048 x 2048 matrices, five
// steps: 1.60 ms, 860 TF/s of symmetric-half flops (1.48 ms cold, before the power
// limit). The tensor pipe is active half of the time: every product, with and without
// C to read, moves its operands at 8 TB/s over all SMs, a chunk in 1980 cycles, where
// its MMAs take 1024 and one SM's copies by themselves 1260 (see Maps).
template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args args) {
  using L = Layout<BN>;
  constexpr int kStages = L::kStages;
  constexpr int kBufs = L::kTmemBufs;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::kBarOff;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kStages + kBufs + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 2 * kBufs);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kMiscOff);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * kNumEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane < args.count) {
    prefetch_tmap(&maps.a[lane]);
    prefetch_tmap(&maps.b[lane]);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  launch_dependents();
  grid_dependency_wait();

  const int num_tiles = args.job[args.count - 1].tile_end;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;
  // Wave k runs the clusters forwards, wave k + 1 backwards: the jobs are
  // sorted by contraction length, so long tiles meet short ones.
  auto tile_of = [&](int k) {
    return k * num_clusters + ((k & 1) ? num_clusters - 1 - cluster_id : cluster_id);
  };
  const int waves = (num_tiles + num_clusters - 1) / num_clusters;
  auto find_job = [&](int& lt) {
    int j = 0;
    while (j + 1 < args.count && lt >= args.job[j].tile_end) ++j;
    if (j > 0) lt -= args.job[j - 1].tile_end;
    return j;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ operand loads
    if (lane == 0) {
      const uint32_t full_leader0 = mapa_shared(full_bar(0), 0);
      uint32_t it = 0;
      bool ok = true;
      for (int k = 0; ok && k < waves; ++k) {
        int lt = tile_of(k);
        if (lt >= num_tiles) continue;
        const int j = find_job(lt);
        int tm, tn;
        tile_at<BN>(args.job[j], lt, tm, tn);
        const int a_row = tm * (2 * BM) + static_cast<int>(rank) * BM;
        const int b_row = tn * BN + static_cast<int>(rank) * (BN / 2);
        const int chunks = args.job[j].chunks;
        const bool a_mn = args.job[j].a_mn != 0, b_mn = args.job[j].b_mn != 0;
        for (int c = 0; c < chunks; ++c, ++it) {
          const int s = it % kStages;
          const uint32_t u = it / kStages;
          if (!mbar_wait(empty_bar(s), (u & 1u) ^ 1u, abort_flag, kErrTimeoutTma)) {
            ok = false;
            break;
          }
          const uint32_t a_dst = sbase + s * L::kStageBytes;
          const uint32_t b_dst = a_dst + L::kABytes;
          const uint32_t fbar = full_leader0 + 8u * s;
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * L::kStageBytes);
          // K-major: rows of the operand, two 64-element blocks of the
          // contraction; MN-major: 128 rows of the contraction, the blocks
          // that hold this CTA's operand rows
          if (a_mn)
            tma_load_3d_pair(a_dst, &maps.a[j], fbar, 0, c * BK, a_row / 64);
          else
            tma_load_3d_pair(a_dst, &maps.a[j], fbar, 0, a_row, 2 * c);
          if (b_mn)
            tma_load_3d_pair(b_dst, &maps.b[j], fbar, 0, c * BK, b_row / 64);
          else
            tma_load_3d_pair(b_dst, &maps.b[j], fbar, 0, b_row, 2 * c);
        }
      }
      if (!ok && leader) {
        for (uint32_t k = 0; k < kStages && k < it; ++k) {
          const uint32_t j = it - 1 - k;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full_bar(j % kStages), (j / kStages) & 1u) &&
                 globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue (even CTA)
    // The whole warp walks the loop, so that addresses and descriptors stay
    // warp-uniform, and one elected lane issues. The next chunk's barrier is
    // probed before this chunk's MMAs are issued: the probe's round trip (about
    // 150 cycles) then runs under the issue instead of adding to it.
    if (leader) {
      const bool elected = elect_one();
      uint32_t it = 0, tc = 0;
      bool ok = true;
      for (int k = 0; ok && k < waves; ++k) {
        int lt = tile_of(k);
        if (lt >= num_tiles) continue;
        const int j = find_job(lt);
        const int chunks = args.job[j].chunks;
        const bool a_mn = args.job[j].a_mn != 0, b_mn = args.job[j].b_mn != 0;
        const uint32_t idesc = idesc_f16(2 * BM, BN, a_mn, b_mn);
        // K = 16 per instruction: 32 bytes along a K-major row (four to a
        // block), or 16 rows of 128 bytes of an MN-major tile, whose
        // 64-element blocks are 16 KB apart
        const uint64_t ad0 = a_mn ? desc_mnmajor_sw128(sbase, 64 * BK * 2) : desc_kmajor_sw128(sbase);
        const uint64_t bd0 = b_mn ? desc_mnmajor_sw128(sbase + L::kABytes, 64 * BK * 2)
                                  : desc_kmajor_sw128(sbase + L::kABytes);
        const uint64_t as = a_mn ? (16 * 128) >> 4 : 32 >> 4;
        const uint64_t bs = b_mn ? (16 * 128) >> 4 : 32 >> 4;
        const uint64_t ah = (a_mn ? 4 * 16 * 128 : L::kABytes / 2) >> 4;   // to the second half
        const uint64_t bh = (b_mn ? 4 * 16 * 128 : L::kBBytes / 2) >> 4;
        const int tb = tc % kBufs;
        const uint32_t tu = tc / kBufs;
        ++tc;
        if (!mbar_wait(tempty_bar(tb), (tu & 1u) ^ 1u, abort_flag, kErrTimeoutMma)) {
          ok = false;
          break;
        }
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(tb * BN);
        bool ready = false;
        for (int c = 0; c < chunks; ++c, ++it) {
          const int s = it % kStages;
          if (!ready && !mbar_wait(full_bar(s), (it / kStages) & 1u, abort_flag, kErrTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t nx = it + 1;
          ready = c + 1 < chunks && mbar_try_wait(full_bar(nx % kStages), (nx / kStages) & 1u);
          const uint64_t off = static_cast<uint64_t>(s * L::kStageBytes) >> 4;
          const uint64_t ad = ad0 + off, bd = bd0 + off;
          if (elected) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_f16_pair(d_tmem, ad + (kk >> 2) * ah + (kk & 3) * as,
                           bd + (kk >> 2) * bh + (kk & 3) * bs, idesc, c > 0 || kk > 0 ? 1u : 0u);
            mma_commit_pair(empty_bar(s), 0x3);
          }
          __syncwarp();
        }
        if (ok && elected) mma_commit_pair(tfull_bar(tb), 0x3);
        __syncwarp();
      }
      if (!ok && elected) {
        mma_commit_pair(drain_bar, 0x1);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
      __syncwarp();
    }
  } else if (warp >= kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                 // TMEM lane quarter: 32 rows
    const int ew = warp - kFirstEpiWarp;
    const int hh = ew >> 2;                 // column half of the tile
    constexpr int kBoxes = BN / 2 / 32;
    const uint32_t slot = sbase + L::kSlotOff + ew * L::kSlotBytes;
    const uint32_t tempty_leader0 = mapa_shared(tempty_bar(0), 0);
    uint32_t tc = 0;
    for (int k = 0; k < waves; ++k) {
      int lt = tile_of(k);
      if (lt >= num_tiles) continue;
      const int j = find_job(lt);
      int tm, tn;
      tile_at<BN>(args.job[j], lt, tm, tn);
      const Job& job = args.job[j];
      const int rows = job.rows, cols = job.cols;
      const int y0 = tm * (2 * BM) + static_cast<int>(rank) * BM + q * 32;
      const int x0 = tn * BN + hh * (BN / 2);
      const bool mirror = job.sym && tn * BN >= (tm + 1) * (2 * BM);
      const bool split = job.split, bf16 = job.bf16;
      const uint16_t* cp = job.c;
      const uint16_t* cp2 = job.c2;
      const float alpha = job.alpha, beta = job.beta, beta2 = job.beta2, diag = job.diag;
      // boxes of this warp that hold anything
      const int boxes = y0 < rows && x0 < cols ? min(kBoxes, (cols - x0 + 31) / 32) : 0;
      // C of box gi, loaded a box ahead (the first one under the tile's products):
      // eight rows of 64 bytes per instruction; lanes get their rows through the
      // staging buffer
      uint4 ch[4], cl[4];
      auto load_c = [&](int gi) {
        const int64_t at = static_cast<int64_t>(y0 + (lane >> 2)) * job.pitch + x0 + gi * 32 +
                           (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = y0 + 8 * i + (lane >> 2) < rows;
          const int64_t e = at + static_cast<int64_t>(8 * i) * job.pitch;
          if (cp != nullptr)
            ch[i] = in ? *reinterpret_cast<const uint4*>(cp + e) : make_uint4(0u, 0u, 0u, 0u);
          if (cp2 != nullptr)
            cl[i] = in ? *reinterpret_cast<const uint4*>(cp2 + e) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      if (boxes > 0) load_c(0);
      const int tb = tc % kBufs;
      const uint32_t tu = tc / kBufs;
      ++tc;
      if (!mbar_wait(tfull_bar(tb), tu & 1u, abort_flag, kErrTimeoutEpi)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(tb * BN + hh * (BN / 2));
      for (int gi = 0; gi < boxes; ++gi) {
        uint32_t r[32];
        tmem_ld32(taddr + gi * 32, r);
        tmem_wait_ld();
        tmem_regs_ready(r);
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]) * alpha;
        __syncwarp();      // the last box has been read
        if (cp != nullptr) {
          put_rows(slot, ch, lane);
          if (cp2 != nullptr) put_rows(slot + L::kBoxBytes, cl, lane);
          if (gi + 1 < boxes) load_c(gi + 1);
          __syncwarp();
          if (cp2 != nullptr) add_scaled(v, slot + L::kBoxBytes, beta2, lane);
          add_scaled(v, slot, beta, lane);
          // a mirror image goes into rows of the second box that other lanes read C2 from
          if (cp2 != nullptr && mirror) __syncwarp();
        }
        if (y0 == x0 + gi * 32) {      // a box on the diagonal
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] -= e == lane ? diag : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {        // 16-byte units of the row's 64 bytes
          const uint32_t at = box_unit(slot, lane, u);
          const float* w = v + 8 * u;
          uint32_t o[4];
          if (bf16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 b2 = __floats2bfloat162_rn(w[2 * e], w[2 * e + 1]);
              o[e] = *reinterpret_cast<uint32_t*>(&b2);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack_f16(w[2 * e], w[2 * e + 1]);
          }
          sts16(at, o[0], o[1], o[2], o[3]);
          if (split) {
            uint32_t l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 hv = unpack_f16(o[e]);
              l[e] = pack_f16((w[2 * e] - hv.x) * kLoScale, (w[2 * e + 1] - hv.y) * kLoScale);
            }
            sts16(at + L::kBoxBytes, l[0], l[1], l[2], l[3]);
          }
          if (mirror) {
            // row = tile column 8u + e, 16-bit position = lane
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int rr = 8 * u + e;
              const uint32_t dst =
                  box_unit(slot + L::kBoxBytes, rr, lane >> 3) + (lane & 7) * 2;
              const uint16_t hv = static_cast<uint16_t>(e & 1 ? o[e >> 1] >> 16 : o[e >> 1]);
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst), "h"(hv) : "memory");
            }
          }
        }
        __syncwarp();
        const int x = x0 + gi * 32;
        store_box(job.out, rows, cols, y0, x, slot, lane);
        if (split) store_box(job.lo, rows, cols, y0, x, slot + L::kBoxBytes, lane);
        if (mirror) store_box(job.out, rows, cols, x, y0, slot + L::kBoxBytes, lane);
      }
      // every TMEM read of this tile has landed
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty_leader0 + 8u * tb);
    }
    // the next launch's copies read what these stores wrote
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }

  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- short sides of up to 256
// With r <= 256 every matrix of the short side is one 256 x 256 tile, and a step's
// products up to P (for a pair of steps, up to P_1 P_0) need nothing from outside the
// pair of CTAs that made A: one launch does them all, a pair of CTAs per job, with the
// matrices in shared memory (each CTA its 128 rows, 64 KB a matrix) and only what
// multiplies X written out. All of them are symmetric, so a CTA's rows are its share
// of both operands, in the Gram product too. Five steps are then 8 launches instead of
// 17 (us: 256 x 768 83 instead of 100, 16 x 256 58 and 79, eight 256 x 1024 99 and 131).
// A product takes 3.4 us: 1.1 of MMAs, 1 for the barriers, 1.4 to read TMEM, round and
// write.
constexpr int kChainDim = 256;
constexpr int kChainOps = 6;            // the Gram product and up to five more

struct ChainJob {
  int r, pitch;                         // rows and row pitch of the result
  int chunks;                           // of the Gram product's contraction
  int last;                             // index of the last product: 1, or 5 for a pair
  int mn;                               // X stored with the contraction outermost
  uint16_t* out;
  float alpha[kChainOps], beta[kChainOps], diag[kChainOps];
  float beta2;                          // of a pair's last product
};
struct ChainArgs {
  ChainJob job[kMaxJobs];
};
struct ChainMaps {
  CUtensorMap x[kMaxJobs];
};

struct ChainLayout {
  static constexpr int kMatrix = BM * kChainDim * 2;          // this CTA's rows of one
  static constexpr int kStageBytes = BM * BK * 2;
  static constexpr int kStages = 2 * kMatrix / kStageBytes;   // where matrices 1 and 2 go later
  static constexpr int kBarOff = 3 * kMatrix;
  static constexpr int kNumBars = 2 * kStages + 4;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kAlloc = kMiscOff + 16 + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

// Product i = 1 .. 5 is alpha a b + beta c, of matrices
//   P_0 = (A_0, A_0; A_0), T = (P_0, A_0; A_0), A_1 = (T, P_0; T), P_1 = (A_1, A_1; A_1),
//   P_1 P_0 (P_0, P_1; P_0 and beta2 P_1)
// kept as A_0, A_1 in 0, P_0 in 1, T and P_1 in 2: four bits per product. The last
// one passes through the matrix that it does not read, 1 (of a step) or 0.
__device__ __forceinline__ int chain_a(int i) { return (0x102100 >> (4 * i)) & 3; }
__device__ __forceinline__ int chain_b(int i) { return (0x201000 >> (4 * i)) & 3; }
__device__ __forceinline__ int chain_c(int i) { return (0x102000 >> (4 * i)) & 3; }
__device__ __forceinline__ int chain_dst(int i) { return (0x020210 >> (4 * i)) & 3; }   // 5: 0

// Byte offset of 16-byte unit u (8 elements) of a CTA's row of a matrix: K-major in
// blocks of 64 columns with the 128-byte swizzle, as an operand of the MMAs.
__device__ __forceinline__ uint32_t chain_unit(int row, int u) {
  return static_cast<uint32_t>((u >> 3) * (BM * 128) + row * 128 + (((u ^ row) & 7) << 4));
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_chain_kernel(const __grid_constant__ ChainMaps maps, const __grid_constant__ ChainArgs args) {
  using L = ChainLayout;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ring = sbase + L::kMatrix;
  const uint32_t bar0 = sbase + L::kBarOff;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  const uint32_t ready_bar = bar0 + 8u * (2 * kStages + 2);   // both CTAs' rows are written
  const uint32_t drain_bar = ready_bar + 8u;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kMiscOff);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int j = static_cast<int>(blockIdx.x >> 1);
  const ChainJob& job = args.job[j];

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar(0), 1);
    mbar_init(tfull_bar(1), 1);
    mbar_init(ready_bar, 2);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    prefetch_tmap(&maps.x[j]);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  launch_dependents();
  grid_dependency_wait();
  const int chunks = job.chunks, last = job.last;

  if (warp == 0) {
    // ------------------------------------------------------------ X, for the Gram product
    if (lane == 0) {
      const uint32_t full_leader0 = mapa_shared(full_bar(0), 0);
      const int row0 = static_cast<int>(rank) * BM;
      const bool mn = job.mn != 0;
      bool ok = true;
      int c = 0;
      for (; c < chunks; ++c) {
        const int s = c % kStages;
        if (!mbar_wait(empty_bar(s), ((c / kStages) & 1u) ^ 1u, abort_flag, kErrTimeoutTma)) {
          ok = false;
          break;
        }
        if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * L::kStageBytes);
        const uint32_t dst = ring + s * L::kStageBytes, bar = full_leader0 + 8u * s;
        if (mn)
          tma_load_3d_pair(dst, &maps.x[j], bar, 0, c * BK, row0 / 64);
        else
          tma_load_3d_pair(dst, &maps.x[j], bar, 0, row0, 2 * c);
      }
      if (!ok && leader) {
        for (int k = 0; k < kStages && k < c; ++k) {
          const int i = c - 1 - k;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full_bar(i % kStages), (i / kStages) & 1u) &&
                 globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue (even CTA)
    if (leader) {
      const bool elected = elect_one();
      const bool mn = job.mn != 0;
      const uint32_t idesc = idesc_f16(2 * BM, kChainDim, mn, mn);
      const uint64_t d0 = mn ? desc_mnmajor_sw128(ring, 64 * BK * 2) : desc_kmajor_sw128(ring);
      const uint64_t ks = mn ? (16 * 128) >> 4 : 32 >> 4;
      const uint64_t kh = (mn ? 4 * 16 * 128 : L::kStageBytes / 2) >> 4;
      bool ok = true;
      for (int c = 0; c < chunks; ++c) {
        const int s = c % kStages;
        if (!mbar_wait(full_bar(s), (c / kStages) & 1u, abort_flag, kErrTimeoutMma)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dd = d0 + (static_cast<uint64_t>(s * L::kStageBytes) >> 4);
        if (elected) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t dk = dd + (kk >> 2) * kh + (kk & 3) * ks;
            mma_f16_pair(tmem_base, dk, dk, idesc, c > 0 || kk > 0 ? 1u : 0u);
          }
          mma_commit_pair(empty_bar(s), 0x3);
        }
        __syncwarp();
      }
      if (ok && elected) mma_commit_pair(tfull_bar(0), 0x3);
      __syncwarp();
      const uint32_t idesc_k = idesc_f16(2 * BM, kChainDim, false, false);
      const int ksteps = (job.r + 15) / 16;
      for (int i = 1; ok && i <= last; ++i) {
        if (!mbar_wait(ready_bar, (i - 1) & 1u, abort_flag, kErrTimeoutMma)) {
          ok = false;
          break;
        }
        // the other CTA's rows were written by its threads
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        tc_fence_after();
        const uint64_t ad = desc_kmajor_sw128(sbase + chain_a(i) * L::kMatrix);
        const uint64_t bd = desc_kmajor_sw128(sbase + chain_b(i) * L::kMatrix);
        if (elected) {
          for (int kk = 0; kk < ksteps; ++kk) {
            const uint64_t off = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
            mma_f16_pair(tmem_base + (i & 1) * kChainDim, ad + off, bd + off, idesc_k,
                         kk > 0 ? 1u : 0u);
          }
          mma_commit_pair(tfull_bar(i & 1), 0x3);
        }
        __syncwarp();
      }
      if (!ok && elected) {
        mma_commit_pair(drain_bar, 0x1);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
      __syncwarp();
    }
  } else if (warp >= kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogues
    const int q = warp & 3, hh = (warp - kFirstEpiWarp) >> 2;
    const int row = q * 32 + lane, grow = static_cast<int>(rank) * BM + row;
    const bool live = grow < job.r;
    const uint32_t ready_leader = mapa_shared(ready_bar, 0);
    for (int i = 0; i <= last; ++i) {
      // (every wait ends; after an expired one all warps of the CTA go on to the
      // barriers below)
      const bool ok = mbar_wait(tfull_bar(i & 1), (i >> 1) & 1u, abort_flag, kErrTimeoutEpi);
      if (__all_sync(0xFFFFFFFFu, ok)) {
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                               static_cast<uint32_t>((i & 1) * kChainDim + hh * 128);
        const uint32_t cm = sbase + chain_c(i) * L::kMatrix;
        const uint32_t dm = sbase + chain_dst(i) * L::kMatrix;
        const float alpha = job.alpha[i], beta = job.beta[i];
        const float diag = live ? job.diag[i] : 0.0f;      // rows past r stay zero
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t acc[32];
          tmem_ld32(taddr + g * 32, acc);
          const int u0 = hh * 16 + g * 4, col0 = u0 * 8;
          uint32_t w[4][4], w2[4][4];
          if (i > 0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) lds16(cm + chain_unit(row, u0 + u), w[u]);
          }
          if (i == kChainOps - 1) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              lds16(sbase + 2 * L::kMatrix + chain_unit(row, u0 + u), w2[u]);
          }
          tmem_wait_ld();
          tmem_regs_ready(acc);
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            fmul2(v[e], v[e + 1], __uint_as_float(acc[e]), __uint_as_float(acc[e + 1]), alpha, alpha);
          if (i == kChainOps - 1) add_scaled(v, w2, job.beta2);
          if (i > 0) add_scaled(v, w, beta);
          if (grow >= col0 && grow < col0 + 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] -= col0 + e == grow ? diag : 0.0f;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack_f16(v[8 * u + 2 * e], v[8 * u + 2 * e + 1]);
            sts16(dm + chain_unit(row, u0 + u), o[0], o[1], o[2], o[3]);
          }
        }
      }
      if (i < last) fence_proxy_async_smem();
      tc_fence_before();
      asm volatile("bar.sync 1, %0;" ::"n"(kNumEpiWarps * 32) : "memory");
      if (i == last) {
        // the result, a row of up to 512 bytes per warp and instruction
        const uint32_t dm = sbase + chain_dst(i) * L::kMatrix;
        if (8 * lane < job.pitch) {
          for (int rr = warp - kFirstEpiWarp; rr < min(BM, job.r - static_cast<int>(rank) * BM);
               rr += kNumEpiWarps) {
            uint32_t o[4];
            lds16(dm + chain_unit(rr, lane), o);
            *reinterpret_cast<uint4*>(
                job.out + static_cast<int64_t>(static_cast<int>(rank) * BM + rr) * job.pitch +
                8 * lane) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        break;
      }
      if (warp == kFirstEpiWarp && lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(ready_leader)
                     : "memory");
    }
    // the next launch's copies read what these stores wrote
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }

  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- input
constexpr int kNormBlocks = 128;       // partial sums of squares per job
constexpr int kSplitThreads = 256;

struct InJob {
  const void* g;        // bf16 or fp32 [rows, cols]
  int64_t count;        // rows * cols, a multiple of 256
  int cols, pitch;      // hi and lo have rows of `pitch` elements
  double* part;         // [kNormBlocks]
  uint16_t* hi;
  uint16_t* lo;
};
struct InArgs {
  InJob job[kMaxJobs];
  int g_f32;
  float eps;
};

__device__ __forceinline__ void load_g8(const void* g, int f32, int64_t i, float (&v)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + i);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
  }
}

// Block sum in 64 bits, the same order every time; the result is in thread 0.
__device__ __forceinline__ double block_sum(double v, double* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += buf[w];
  __syncthreads();
  return s;
}

__global__ void __launch_bounds__(kSplitThreads) ns_sumsq_kernel(const __grid_constant__ InArgs a) {
  __shared__ double buf[kSplitThreads / 32];
  launch_dependents();
  grid_dependency_wait();
  const InJob& j = a.job[blockIdx.y];
  double sum = 0.0;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x) * 8; i < j.count;
       i += static_cast<int64_t>(kNormBlocks) * kSplitThreads * 8) {
    float v[8];
    load_g8(j.g, a.g_f32, i, v);
    // squares of fp32 values far from 1 leave fp32's range: 64 bits
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), sum);
  }
  sum = block_sum(sum, buf);
  if (threadIdx.x == 0) j.part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kSplitThreads) ns_split_kernel(const __grid_constant__ InArgs a) {
  __shared__ double buf[kSplitThreads / 32];
  launch_dependents();
  grid_dependency_wait();
  const InJob& j = a.job[blockIdx.y];
  const double ss = block_sum(threadIdx.x < kNormBlocks ? j.part[threadIdx.x] : 0.0, buf);
  const double scale = kXScale / (sqrt(ss) + static_cast<double>(a.eps));
  const int64_t total = j.count / j.cols * j.pitch;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x) * 8; i < total;
       i += static_cast<int64_t>(gridDim.x) * kSplitThreads * 8) {
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (j.pitch == j.cols) {
      load_g8(j.g, a.g_f32, i, v);
    } else {
      const int64_t row = i / j.pitch;
      const int col = static_cast<int>(i - row * j.pitch);
      if (col < j.cols) load_g8(j.g, a.g_f32, row * j.cols + col, v);
    }
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = static_cast<float>(v[2 * e] * scale), y = static_cast<float>(v[2 * e + 1] * scale);
      h[e] = pack_f16(x, y);
      const float2 f = unpack_f16(h[e]);
      l[e] = pack_f16((x - f.x) * kLoScale, (y - f.y) * kLoScale);
    }
    *reinterpret_cast<uint4*>(j.hi + i) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(j.lo + i) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

}  // namespace ns
}  // namespace fp8bw
