// newton_schulz.cuh -- orthogonalisation of weight updates by Newton-Schulz
// products on the tensor cores (sm_100a, tcgen05 on CTA pairs).
//
//   X_0 = G / (||G||_F + eps)
//   A = X X^T,  B = b A + c A A,  X <- a X + B X          (rows <= columns)
//   A = X^T X,  B = b A + c A A,  X <- a X + X B          (rows >  columns)
// so A and B are r x r with r the shorter side. A step is three launches of
// one GEMM kernel, each over all jobs (matrices) of the call:
//   gram    A, only its tiles on and above the diagonal; each of the others is
//           written as the transpose of its mirror image from the same registers
//   poly    B, likewise (A is symmetric, so A A = A A^T)
//   update  the new X, added to a X in the epilogue
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
constexpr int BK = 64;             // contraction chunk: 128 bytes of fp16
constexpr int kThreads = 384;
constexpr int kFirstEpiWarp = 4;
constexpr int kNumEpiWarps = 8;
constexpr float kXScale = 1024.0f;     // X is stored times this
constexpr float kAScale = 4096.0f;     // A and B are stored times this
constexpr float kLoScale = 2048.0f;    // lo = (x - hi) * this

constexpr int kShiftStep = 3;

enum Mode : int { kGram = 0, kPoly = 1, kUpdate = 2, kLast = 3 };

struct Job {
  int rows, cols;            // output
  int tiles_m, tiles_n;      // 256 x BN tiles
  int chunks;                // of the contraction
  int a_mn, b_mn;            // operand stored with the contraction outermost
  int tile_end;              // cumulative tile count
};

struct Maps {
  CUtensorMap a[kMaxJobs];     // operands
  CUtensorMap b[kMaxJobs];
  CUtensorMap c[kMaxJobs];     // poly: A; update, last: the old hi  (32 x 32 boxes)
  CUtensorMap lo[kMaxJobs];    // update, last: lo
  CUtensorMap out[kMaxJobs];   // the result
};

struct Args {
  Job job[kMaxJobs];
  int count;
  float alpha, beta;           // result = alpha * product + beta * C
  float diag;                  // poly: minus this on the diagonal
};

template <int BN_>
struct Layout {
  static constexpr int BN = BN_;
  static constexpr int kStages = BN == 256 ? 4 : 5;
  static constexpr int kTmemBufs = 512 / BN;
  static constexpr int kABytes = BM * BK * 2;
  static constexpr int kBBytes = (BN / 2) * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kSlots = 3;                 // C / result boxes per warp
  static constexpr int kAhead = kSlots - 1;        // C boxes requested ahead
  static constexpr int kBoxBytes = 32 * 32 * 2;
  static constexpr int kSlotBytes = 2 * kBoxBytes;
  static constexpr int kSlotOff = kRingBytes;
  static constexpr int kBarOff = kSlotOff + kNumEpiWarps * kSlots * kSlotBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kTmemBufs + 1 + kNumEpiWarps * kSlots;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kBytes = kMiscOff + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

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

// Tile `lt` of a job -> (tm, tn). Symmetric results (SYM) number only the
// tiles that reach the diagonal's 256-row block or lie right of it.
template <int BN, bool SYM>
__device__ __forceinline__ void tile_at(int lt, int tiles_n, int& tm, int& tn) {
  if constexpr (SYM) {
    constexpr int kPer = 256 / BN;
    tm = 0;
    int left = tiles_n;
    while (lt >= left) {
      lt -= left;
      left -= kPer;
      ++tm;
    }
    tn = tm * kPer + lt;
  } else {
    tm = lt / tiles_n;
    tn = lt - tm * tiles_n;
  }
}

// Output tiles of 256 x BN by clusters of two CTAs, each CTA holding 128 rows
// of A and BN/2 rows of B per chunk; roles as in the blockwise GEMMs: warp 0
// loads operands, warp 1 of the even CTA issues the MMAs, warps 4-11 read TMEM
// and write the result box by box (32 x 32) through shared memory and TMA. The
// product of a whole tile stays in TMEM (512 / BN tiles fit), so the epilogue
// of one tile runs under the MMAs of the next.
template <int BN, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args args) {
  using L = Layout<BN>;
  constexpr int kStages = L::kStages;
  constexpr int kBufs = L::kTmemBufs;
  constexpr bool kSym = MODE == kGram || MODE == kPoly;
  constexpr bool kHasC = MODE != kGram;
  constexpr bool kHasLo = MODE == kUpdate || MODE == kLast;

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
  auto slot_bar = [&](int w, int s) { return drain_bar + 8u * (1 + w * L::kSlots + s); };
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
    for (int i = 0; i < kNumEpiWarps * L::kSlots; ++i) mbar_init(slot_bar(0, i), 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane < args.count) {
    prefetch_tmap(&maps.a[lane]);
    prefetch_tmap(&maps.b[lane]);
    prefetch_tmap(&maps.out[lane]);
    if (kHasC) prefetch_tmap(&maps.c[lane]);
    if (kHasLo) prefetch_tmap(&maps.lo[lane]);
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
        tile_at<BN, kSym>(lt, args.job[j].tiles_n, tm, tn);
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
          if (a_mn) {
            tma_load_2d_pair(a_dst, &maps.a[j], fbar, a_row, c * BK);
            tma_load_2d_pair(a_dst + 64 * BK * 2, &maps.a[j], fbar, a_row + 64, c * BK);
          } else {
            tma_load_2d_pair(a_dst, &maps.a[j], fbar, c * BK, a_row);
          }
          if (b_mn) {
            tma_load_2d_pair(b_dst, &maps.b[j], fbar, b_row, c * BK);
            if constexpr (BN == 256)
              tma_load_2d_pair(b_dst + 64 * BK * 2, &maps.b[j], fbar, b_row + 64, c * BK);
          } else {
            tma_load_2d_pair(b_dst, &maps.b[j], fbar, c * BK, b_row);
          }
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
        // K = 16 per instruction: 32 bytes along a K-major row, or 16 rows
        // of 128 bytes of an MN-major tile (64-element atoms 8 KB apart)
        const uint64_t ad0 = a_mn ? desc_mnmajor_sw128(sbase, 64 * BK * 2) : desc_kmajor_sw128(sbase);
        const uint64_t bd0 = b_mn ? desc_mnmajor_sw128(sbase + L::kABytes, 64 * BK * 2)
                                  : desc_kmajor_sw128(sbase + L::kABytes);
        const uint64_t as = a_mn ? (16 * 128) >> 4 : 32 >> 4;
        const uint64_t bs = b_mn ? (16 * 128) >> 4 : 32 >> 4;
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
              mma_f16_pair(d_tmem, ad + kk * as, bd + kk * bs, idesc, c > 0 || kk > 0 ? 1u : 0u);
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
    const uint32_t slot0 = sbase + L::kSlotOff + ew * L::kSlots * L::kSlotBytes;
    const uint32_t tempty_leader0 = mapa_shared(tempty_bar(0), 0);
    uint32_t tc = 0;
    uint32_t loads = 0, used = 0;           // C boxes requested / consumed
    uint32_t stores = 0;                    // result boxes written (no C)
    bool ok = true;
    for (int k = 0; ok && k < waves; ++k) {
      int lt = tile_of(k);
      if (lt >= num_tiles) continue;
      const int j = find_job(lt);
      int tm, tn;
      tile_at<BN, kSym>(lt, args.job[j].tiles_n, tm, tn);
      const int rows = args.job[j].rows, cols = args.job[j].cols;
      const int y0 = tm * (2 * BM) + static_cast<int>(rank) * BM + q * 32;
      const int x0 = tn * BN + hh * (BN / 2);
      const bool mirror = kSym && tn * BN >= (tm + 1) * (2 * BM);
      // boxes of this warp that hold anything
      const int boxes = y0 < rows && x0 < cols ? min(kBoxes, (cols - x0 + 31) / 32) : 0;
      // C of box gi into the next slot; before that, the stores that used the
      // slot must have read it
      auto load_c = [&](int gi) {
        const int s = loads % L::kSlots;
        if (lane == 0) {
          bulk_wait_group_read<L::kSlots - L::kAhead>();
          const uint32_t dst = slot0 + s * L::kSlotBytes;
          mbar_arrive_expect_tx(slot_bar(ew, s), kHasLo ? 2 * L::kBoxBytes : L::kBoxBytes);
          tma_load_2d(dst, &maps.c[j], slot_bar(ew, s), x0 + gi * 32, y0);
          if constexpr (kHasLo)
            tma_load_2d(dst + L::kBoxBytes, &maps.lo[j], slot_bar(ew, s), x0 + gi * 32, y0);
        }
        ++loads;
      };
      if constexpr (kHasC) {
        if (boxes > 0) {
          if (lane == 0) bulk_wait_group_read<0>();
          for (int gi = 0; gi < L::kAhead && gi < boxes; ++gi) load_c(gi);
        }
      }
      const int tb = tc % kBufs;
      const uint32_t tu = tc / kBufs;
      ++tc;
      if (!mbar_wait(tfull_bar(tb), tu & 1u, abort_flag, kErrTimeoutEpi)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(tb * BN + hh * (BN / 2));
      for (int gi = 0; gi < boxes; ++gi) {
        uint32_t r[32];
        tmem_ld32(taddr + gi * 32, r);
        uint32_t slot;
        if constexpr (kHasC) {
          const int s = used % L::kSlots;
          if (!mbar_wait(slot_bar(ew, s), (used / L::kSlots) & 1u, abort_flag, kErrTimeoutEpi)) {
            ok = false;
            break;
          }
          ++used;
          slot = slot0 + s * L::kSlotBytes;
        } else {
          slot = slot0 + (stores % L::kSlots) * L::kSlotBytes;
          ++stores;
          if (lane == 0) bulk_wait_group_read<L::kSlots - 1>();
          __syncwarp();
        }
        tmem_wait_ld();
        tmem_regs_ready(r);
#pragma unroll
        for (int u = 0; u < 4; ++u) {        // 16-byte units of the row's 64 bytes
          const uint32_t at = slot + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4);
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[8 * u + e]) * args.alpha;
          if constexpr (kHasC) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(at)
                         : "memory");
            float c[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack_f16(w[e]);
              c[2 * e] = f.x;
              c[2 * e + 1] = f.y;
            }
            if constexpr (kHasLo) {
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                           : "r"(at + L::kBoxBytes)
                           : "memory");
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack_f16(w[e]);
                c[2 * e] = fmaf(f.x, 1.0f / kLoScale, c[2 * e]);
                c[2 * e + 1] = fmaf(f.y, 1.0f / kLoScale, c[2 * e + 1]);
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(args.beta, c[e], v[e]);
            if constexpr (MODE == kPoly) {
              if (y0 == x0 + gi * 32) {      // a box on the diagonal
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] -= 8 * u + e == lane ? args.diag : 0.0f;
              }
            }
          }
          uint32_t o[4];
          if constexpr (MODE == kLast) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
              o[e] = *reinterpret_cast<uint32_t*>(&b2);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack_f16(v[2 * e], v[2 * e + 1]);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[0]), "r"(o[1]),
                       "r"(o[2]), "r"(o[3])
                       : "memory");
          if constexpr (MODE == kUpdate) {
            uint32_t l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 hv = unpack_f16(o[e]);
              l[e] = pack_f16((v[2 * e] - hv.x) * kLoScale, (v[2 * e + 1] - hv.y) * kLoScale);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + L::kBoxBytes),
                         "r"(l[0]), "r"(l[1]), "r"(l[2]), "r"(l[3])
                         : "memory");
          }
          if constexpr (kSym) {
            if (mirror) {
              // row = tile column 8u + e, 16-bit position = lane
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int rr = 8 * u + e;
                const uint32_t dst = slot + L::kBoxBytes + rr * 64 +
                                     (((lane >> 3) ^ ((rr >> 1) & 3)) << 4) + (lane & 7) * 2;
                const uint16_t hv = static_cast<uint16_t>(e & 1 ? o[e >> 1] >> 16 : o[e >> 1]);
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst), "h"(hv) : "memory");
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&maps.out[j], slot, x0 + gi * 32, y0);
          if constexpr (MODE == kUpdate) tma_store_2d(&maps.lo[j], slot + L::kBoxBytes, x0 + gi * 32, y0);
          if constexpr (kSym) {
            if (mirror) tma_store_2d(&maps.out[j], slot + L::kBoxBytes, y0, x0 + gi * 32);
          }
          bulk_commit_group();
        }
        if constexpr (kHasC) {
          if (gi + L::kAhead < boxes) load_c(gi + L::kAhead);
        }
      }
      if (!ok) break;
      // every TMEM read of this tile has landed
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty_leader0 + 8u * tb);
    }
    if (lane == 0) {
      for (; used < loads; ++used) {     // after an expired wait: let the copies land
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(slot_bar(ew, used % L::kSlots), (used / L::kSlots) & 1u) &&
               globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
      bulk_wait_group_all();
    }
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
  const void* g;        // bf16 or fp32, count elements (a multiple of 256)
  int64_t count;
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
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x) * 8; i < j.count;
       i += static_cast<int64_t>(gridDim.x) * kSplitThreads * 8) {
    float v[8];
    load_g8(j.g, a.g_f32, i, v);
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
