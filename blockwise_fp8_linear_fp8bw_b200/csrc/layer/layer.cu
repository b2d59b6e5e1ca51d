// layer.cu -- the C ABI of the layer operators (declared in
// include/fp8bw_layer.h): argument checks, TMA descriptors, launches. Its own
// translation unit, with its own device error record.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../../include/fp8bw_layer.h"
#include "../common.cuh"
#include "newton_schulz.cuh"
#include "norm.cuh"
#include "swiglu.cuh"

namespace fp8bw {
namespace layer {
namespace {

// ---------------------------------------------------------------- device, checks
struct Device {
  int ordinal = 0;
  int sm_count = 0;
};

int current_device(Device* out) {
  struct Info {
    int checked = 0;   // 0 = unknown, 1 = sm_100, -1 = other
    int sms = 0;
  };
  static Info info[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return FP8BW_ERR_DEVICE;
  // makes the primary context current on this thread (the tensor-map encoder
  // needs one)
  if (cudaSetDevice(dev) != cudaSuccess) return FP8BW_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  Info& d = info[dev];
  if (d.checked == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return FP8BW_ERR_DEVICE;
    d.checked = (major == 10 && minor == 0) ? 1 : -1;
  }
  if (d.checked != 1) return FP8BW_ERR_DEVICE;
  out->ordinal = dev;
  out->sm_count = d.sms;
  return FP8BW_OK;
}

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxNormCols = 32768;    // a row fits 512 threads x 8 chunks
constexpr int64_t kMaxGluCols = int64_t(1) << 22;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t pad16(int64_t rows) { return (rows + 15) / 16 * 16; }
bool cols_ok(int64_t c, int64_t most) { return c >= 0 && c % 16 == 0 && c <= most; }

// The buffers of a call: each is checked for presence and alignment, and
// every output against every other buffer.
struct Buffers {
  struct Item {
    uintptr_t lo, hi;
    bool out;
  };
  Item item[32];
  int n = 0;
  int status = FP8BW_OK;
  void add(const void* p, int64_t bytes, bool required, bool out) {
    if (status != FP8BW_OK) return;
    if (p == nullptr) {
      if (required && bytes > 0) status = FP8BW_ERR_NULL;
      return;
    }
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a % 16 != 0) {
      status = FP8BW_ERR_ALIGN;
      return;
    }
    if (bytes <= 0) return;
    if (n == static_cast<int>(sizeof item / sizeof item[0])) {
      status = FP8BW_ERR_SHAPE;
      return;
    }
    item[n++] = Item{a, a + static_cast<uintptr_t>(bytes), out};
  }
  void in(const void* p, int64_t bytes, bool required = true) { add(p, bytes, required, false); }
  void out(const void* p, int64_t bytes, bool required = true) { add(p, bytes, required, true); }
  int check() const {
    if (status != FP8BW_OK) return status;
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j)
        if ((item[i].out || item[j].out) && item[i].lo < item[j].hi && item[j].lo < item[i].hi)
          return FP8BW_ERR_ALIAS;
    return FP8BW_OK;
  }
};

int launched(cudaError_t e) {
  if (e != cudaSuccess) return FP8BW_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? FP8BW_OK : FP8BW_ERR_LAUNCH;
}

// ---------------------------------------------------------------- tensor maps
int tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* out) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (encode == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || p == nullptr)
      return FP8BW_ERR_CUDA;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  *out = encode;
  return FP8BW_OK;
}

// bf16 [rows, cols] with rows of row_bytes, read in 128 x 128 tiles.
int encode_tiles(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                 int64_t row_bytes) {
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  const int st = tensor_map_encoder(&encode);
  if (st != FP8BW_OK) return st;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {kTile, kTile};
  const cuuint32_t estr[2] = {1u, 1u};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? FP8BW_OK
             : FP8BW_ERR_CUDA;
}

template <typename K>
int allow_smem(DevicePrep& prep, int dev, K kernel, int bytes) {
  int unused = 0;
  return prepare_for_device(prep, dev, &unused, [&](int*) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
                   cudaSuccess
               ? static_cast<int>(FP8BW_OK)
               : static_cast<int>(FP8BW_ERR_LAUNCH);
  });
}

// ---------------------------------------------------------------- norm
int threads_per_row(int64_t chunks, int v) { return static_cast<int>(cdiv(cdiv(chunks, v), 32) * 32); }

template <int V, int R, bool POW2>
int launch_norm_rows(NormArgs a, cudaStream_t stream) {
  a.tpr = threads_per_row(a.cols / 8, V);
  const int groups = std::max(1, 256 / a.tpr);
  const int64_t blocks = cdiv(a.rows_pad, groups * R);
  const auto kernel = a.cols == 8 * static_cast<int64_t>(V) * a.tpr
                          ? rmsnorm_row_kernel<V, R, true, POW2>
                          : rmsnorm_row_kernel<V, R, false, POW2>;
  return launched(launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(groups * a.tpr),
                                0, stream, a));
}

template <bool POW2>
int norm_rows(const NormArgs& a, const Device& dev, cudaStream_t stream) {
  const int64_t chunks = a.cols / 8;
  // Chunks per thread: one while there are no more than 512 threads' worth of them
  // per SM (latency: 1 x 2048 2.1 us with one, 2.4 with two, 2.7 with four; 200 x
  // 2048 2.5, 2.7, 3.2), two up to 1024 (512 x 2048 3.9, 3.4, 3.8), then four, for
  // loads in flight: as two chunks of two rows, which leaves fewer threads idle than
  // four of one row (16384 x 2048 39.1 and 39.6 us, 45.8 with one chunk and 39.9 with
  // eight; 16384 x 1040 24.5, 27.4, 29.6), of one row where a block would have to be
  // larger (4096 x 8192 41.3, 40.4), and one of four rows in short ones (16384 x 128
  // 6.6, 10.8, 5.1). Rows of more than 512 chunks never have one (148 x 8192 5.4, 3.9
  // with two, 4.1 with four).
  const int64_t total = a.rows_pad * chunks;
  if (total > 1024 * dev.sm_count) {
    if (chunks <= 32) return launch_norm_rows<1, 4, POW2>(a, stream);
    if (chunks <= 512) return launch_norm_rows<2, 2, POW2>(a, stream);
  } else {
    if (total <= 512 * dev.sm_count && chunks <= 512) return launch_norm_rows<1, 1, POW2>(a, stream);
    if (chunks <= 1024) return launch_norm_rows<2, 1, POW2>(a, stream);
  }
  if (chunks <= 2048) return launch_norm_rows<4, 1, POW2>(a, stream);
  return launch_norm_rows<8, 1, POW2>(a, stream);
}

template <bool POW2>
int rmsnorm_quantize(const uint16_t* x, const uint16_t* residual, const void* gamma,
                     int gamma_is_f32, int64_t rows, int64_t cols, float eps, uint16_t* h,
                     float* rstd, uint16_t* y, uint8_t* q, float* s, uint8_t* q_t, float* s_t,
                     void* stream) {
  if (rows < 0 || rows > kMaxRows || !cols_ok(cols, kMaxNormCols)) return FP8BW_ERR_SHAPE;
  if (q_t != nullptr && cdiv(rows, 128) * cdiv(cols, kColTile) > INT32_MAX)
    return FP8BW_ERR_SHAPE;
  if (!(eps >= 0.0f)) return FP8BW_ERR_SHAPE;
  const int64_t rp = pad16(rows), n = rows * cols;
  if (n > 0 && ((q == nullptr) != (s == nullptr) || (q_t == nullptr) != (s_t == nullptr)))
    return FP8BW_ERR_NULL;
  if (n > 0 && residual == nullptr && h != nullptr) return FP8BW_ERR_NULL;
  Buffers b;
  b.in(x, 2 * n);
  b.in(residual, 2 * n, false);
  b.in(gamma, cols * (gamma_is_f32 ? 4 : 2));
  b.out(h, 2 * n, residual != nullptr);
  b.out(rstd, 4 * rows, q_t != nullptr);
  b.out(y, 2 * n, false);
  b.out(q, rp * cols, false);
  b.out(s, 4 * cdiv(cols, 128) * rp, false);
  b.out(q_t, rp * cols, false);
  b.out(s_t, 4 * cdiv(rp, 128) * cols, false);
  int st = b.check();
  if (st != FP8BW_OK) return st;
  Device dev;
  st = current_device(&dev);
  if (st != FP8BW_OK || n == 0) return st;

  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.gamma_f32 = gamma_is_f32 != 0;
  a.rows = rows;
  a.rows_pad = rp;
  a.cols = cols;
  a.inv_cols = 1.0 / static_cast<double>(cols);
  a.eps = eps;
  a.h = h;
  a.rstd = rstd;
  a.y = y;
  a.q = q;
  a.s = s;
  st = norm_rows<POW2>(a, dev, cs);
  if (st != FP8BW_OK || q_t == nullptr) return st;
  NormColArgs c{};
  c.h = residual != nullptr ? h : x;
  c.rstd = rstd;
  c.gamma = gamma;
  c.gamma_f32 = a.gamma_f32;
  c.rows = rows;
  c.rows_pad = rp;
  c.cols = cols;
  c.tiles_r = static_cast<int>(cdiv(rp, 128));
  c.tiles_c = static_cast<int>(cdiv(cols, kColTile));
  c.q_t = q_t;
  c.s_t = s_t;
  const int64_t tiles = static_cast<int64_t>(c.tiles_r) * c.tiles_c;
  return launched(launch_kernel(norm_col_kernel<POW2>, dim3(static_cast<unsigned>(tiles)),
                                dim3(kColThreads), 0, cs, c));
}

// ---------------------------------------------------------------- norm, backward
constexpr int64_t kBwdSms = 148;      // (the workspace's size must not ask the device)
constexpr int kBwdSmThreads = 512;    // of 128 registers

struct BwdPlan {
  int v, r, tpr, groups, per_sm;
  int64_t blocks;
};

// Chunks of a row per thread that fit it into 512 threads; up to 512 chunks the
// choice of one chunk of two rows or two of one that has more of them on an SM, the
// next ones loading meanwhile (16384 x 2064: 258 chunks, one block of 288 threads per
// SM or three of 160). Blocks of about 128 threads or a row, as many as an SM's
// registers hold (16384 x 1040, 160 threads: 30.4 us with three per SM, 36.2 with
// two; 16384 x 528 18.9 and with 256 threads 20.0), but no more than the iterations
// need: a partial sum costs the last kernel time (1037 x 1040: 6.3 us with 260 of
// them, 7.3 with 444).
BwdPlan bwd_plan(int64_t rows, int64_t cols) {
  const int64_t chunks = cols / 8;
  auto plan = [&](int v) {
    BwdPlan p;
    p.v = v;
    p.r = v == 1 ? 2 : 1;
    p.tpr = threads_per_row(chunks, v);
    // (the kernel adds the groups' partial sums up with one chunk per thread only)
    p.groups = v == 1 ? std::max(1, 128 / std::max(p.tpr, 1)) : 1;
    p.per_sm = std::max(1, kBwdSmThreads / std::max(p.groups * p.tpr, 1));
    return p;
  };
  auto in_flight = [](const BwdPlan& p) { return p.per_sm * p.groups * p.r; };   // rows
  BwdPlan p = plan(chunks <= 512 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8);
  if (p.v == 1 && in_flight(plan(2)) > in_flight(p)) p = plan(2);
  const int64_t steps = cdiv(rows, static_cast<int64_t>(p.groups) * p.r);
  p.blocks = cdiv(steps, std::max<int64_t>(1, cdiv(steps, kBwdSms * p.per_sm)));
  return p;
}

int rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const float* rstd, const void* gamma,
                     int gamma_is_f32, const uint16_t* dres, int64_t rows, int64_t cols,
                     uint16_t* dh, float* dgamma, void* ws, int64_t ws_bytes, void* stream) {
  if (rows < 0 || rows > kMaxRows || !cols_ok(cols, kMaxNormCols)) return FP8BW_ERR_SHAPE;
  const int64_t n = rows * cols;
  const int64_t need = n > 0 ? bwd_plan(rows, cols).blocks * cols * 4 : 0;
  if (ws_bytes < need) return FP8BW_ERR_SHAPE;
  Buffers b;
  b.in(dy, 2 * n);
  b.in(h, 2 * n);
  b.in(rstd, 4 * rows);
  b.in(gamma, cols * (gamma_is_f32 ? 4 : 2), n > 0);
  b.in(dres, 2 * n, false);
  b.out(dh, 2 * n);
  b.out(dgamma, 4 * cols);
  b.out(ws, need);
  int st = b.check();
  if (st != FP8BW_OK) return st;
  Device dev;
  st = current_device(&dev);
  if (st != FP8BW_OK || cols == 0) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (rows == 0)      // a sum over no rows
    return cudaMemsetAsync(dgamma, 0, static_cast<size_t>(cols) * 4, cs) == cudaSuccess
               ? FP8BW_OK
               : FP8BW_ERR_CUDA;
  const BwdPlan p = bwd_plan(rows, cols);
  NormBwdArgs a{dy, h, rstd, gamma, gamma_is_f32 != 0, dres, rows, cols, dh,
                static_cast<float*>(ws), p.tpr};
  using Kernel = void (*)(NormBwdArgs);
  const Kernel kernel = p.v == 1   ? rmsnorm_bwd_kernel<1, 2>
                        : p.v == 2 ? rmsnorm_bwd_kernel<2, 1>
                        : p.v == 4 ? rmsnorm_bwd_kernel<4, 1>
                                   : rmsnorm_bwd_kernel<8, 1>;
  st = launched(launch_kernel(kernel, dim3(static_cast<unsigned>(p.blocks)),
                              dim3(p.groups * p.tpr), 0, cs, a));
  if (st != FP8BW_OK) return st;
  // Eight columns per block where 32 would leave few blocks with long slices (us, with
  // 8 and with 32: 1907 x 128 4.5 and 5.5, 778 x 320 4.7 and 5.8, 933 x 944 6.5 and
  // 7.2, 16384 x 1040 30.4 and 31.3; but 1037 x 1040, of 260 sums, 6.6 and 6.4)
  const float* part = static_cast<const float*>(ws);
  if (cols <= (p.blocks > 288 ? 2048 : 1024))
    return launched(launch_kernel(dgamma_reduce_kernel<8>, dim3(static_cast<unsigned>(cdiv(cols, 8))),
                                  dim3(1024), 0, cs, part, p.blocks, cols, dgamma));
  return launched(launch_kernel(dgamma_reduce_kernel<32>, dim3(static_cast<unsigned>(cdiv(cols, 32))),
                                dim3(1024), 0, cs, part, p.blocks, cols, dgamma));
}

// ---------------------------------------------------------------- gated product
bool glu_shape_ok(int64_t rows, int64_t f) {
  return rows >= 0 && rows <= kMaxRows && cols_ok(f, kMaxGluCols) &&
         cdiv(rows, 128) * cdiv(2 * f, 128) <= INT32_MAX;
}

// 128 x 128 tiles of an output (they fit 31 bits: glu_shape_ok)
int glu_tiles(const CodesOut& out) {
  return static_cast<int>(cdiv(out.rows, kTile) * cdiv(out.cols, kTile));
}

template <bool POW2, bool BWD>
int launch_glu_few(const uint16_t* gu, const uint16_t* da, int64_t rows, int64_t f,
                   const CodesOut& out, cudaStream_t stream) {
  const int64_t row_blocks = out.rows / 16 * cdiv(out.cols, kTile);
  const int64_t tiles_c = cdiv(out.cols, kColTile);
  const int64_t tiles = cdiv(out.rows, kTile) * tiles_c;
  const GluFewArgs a{gu, da, rows, f, out, static_cast<int>(row_blocks), static_cast<int>(tiles_c)};
  return launched(launch_kernel(swiglu_few_kernel<POW2, BWD>,
                                dim3(static_cast<unsigned>(row_blocks + tiles)), dim3(kColThreads),
                                0, stream, a));
}

template <bool POW2>
int swiglu_quantize(const uint16_t* gu, int64_t rows, int64_t f, uint8_t* q, float* s,
                    uint8_t* q_t, float* s_t, void* stream) {
  if (!glu_shape_ok(rows, f)) return FP8BW_ERR_SHAPE;
  const int64_t rp = pad16(rows), n = rows * f;
  if (n > 0 && (q_t == nullptr) != (s_t == nullptr)) return FP8BW_ERR_NULL;
  Buffers b;
  b.in(gu, 4 * n);
  b.out(q, rp * f);
  b.out(s, 4 * cdiv(f, 128) * rp);
  b.out(q_t, rp * f, false);
  b.out(s_t, 4 * cdiv(rp, 128) * f, false);
  int st = b.check();
  if (st != FP8BW_OK) return st;
  Device dev;
  st = current_device(&dev);
  if (st != FP8BW_OK || n == 0) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const CodesOut out{q, s, q_t, s_t, rp, f};
  if (q_t == nullptr)
    return launched(launch_kernel(swiglu_row_kernel<POW2>,
                                  dim3(static_cast<unsigned>(rp / 16),
                                       static_cast<unsigned>(cdiv(f, 128))),
                                  dim3(kColThreads), 0, cs, GluFewArgs{gu, nullptr, rows, f, out}));
  if (glu_tiles(out) <= dev.sm_count)
    return launch_glu_few<POW2, false>(gu, nullptr, rows, f, out, cs);
  CUtensorMap mg, mu;
  st = encode_tiles(&mg, gu, rows, f, 4 * f);
  if (st == FP8BW_OK) st = encode_tiles(&mu, gu + f, rows, f, 4 * f);
  if (st != FP8BW_OK) return st;
  static DevicePrep prep;
  st = allow_smem(prep, dev.ordinal, swiglu_tile_kernel<POW2>, GluFwdSmem::kAlloc);
  if (st != FP8BW_OK) return st;
  const GluTileArgs a{static_cast<int>(cdiv(rp, 128)), static_cast<int>(cdiv(f, 128)),
                      out};
  const int tiles = a.tiles_r * ((a.tiles_c + 1) / 2);     // pairs
  return launched(launch_kernel(swiglu_tile_kernel<POW2>, dim3(std::min(tiles, dev.sm_count)),
                                dim3(kTileThreads), GluFwdSmem::kAlloc, cs, mg, mu, a));
}

template <bool POW2>
int swiglu_backward_quantize(const uint16_t* da, const uint16_t* gu, int64_t rows, int64_t f,
                             uint8_t* q, float* s, uint8_t* q_t, float* s_t, void* stream) {
  if (!glu_shape_ok(rows, f)) return FP8BW_ERR_SHAPE;
  const int64_t rp = pad16(rows), n = rows * f;
  Buffers b;
  b.in(da, 2 * n);
  b.in(gu, 4 * n);
  b.out(q, 2 * rp * f);
  b.out(s, 4 * cdiv(2 * f, 128) * rp);
  b.out(q_t, 2 * rp * f);
  b.out(s_t, 4 * cdiv(rp, 128) * 2 * f);
  int st = b.check();
  if (st != FP8BW_OK) return st;
  Device dev;
  st = current_device(&dev);
  if (st != FP8BW_OK || n == 0) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int tiles_r = static_cast<int>(cdiv(rp, 128)), tiles_c = static_cast<int>(cdiv(f, 128));
  const dim3 grid(std::min(tiles_r * tiles_c, dev.sm_count)), block(kTileThreads);
  const CodesOut out{q, s, q_t, s_t, rp, 2 * f};
  static DevicePrep prep[2];
  if (glu_tiles(out) <= dev.sm_count)
    return launch_glu_few<POW2, true>(gu, da, rows, f, out, cs);
  if (f % 128 != 0 && glu_tiles(out) <= 2 * dev.sm_count) {
    const GluRaggedArgs r{gu, da, rows, f,
                          GluTileArgs{tiles_r, static_cast<int>(cdiv(2 * f, 128)), out}};
    return launched(launch_kernel(swiglu_bwd_ragged_kernel<POW2>, dim3(glu_tiles(out)), block,
                                  TileEmit<1, false>::kBytes + 128, cs, r));
  }
  CUtensorMap mg, mu, md;
  st = encode_tiles(&mg, gu, rows, f, 4 * f);
  if (st == FP8BW_OK) st = encode_tiles(&mu, gu + f, rows, f, 4 * f);
  if (st == FP8BW_OK) st = encode_tiles(&md, da, rows, f, 2 * f);
  if (st != FP8BW_OK) return st;
  if (f % 128 != 0) {
    st = allow_smem(prep[1], dev.ordinal, swiglu_bwd_shift_kernel<POW2>, GluShiftSmem::kAlloc);
    if (st != FP8BW_OK) return st;
    const GluShiftArgs a{gu, da, rows, static_cast<int>(f), tiles_r, out};
    return launched(launch_kernel(swiglu_bwd_shift_kernel<POW2>, grid, block, GluShiftSmem::kAlloc,
                                  cs, mg, mu, md, a));
  }
  st = allow_smem(prep[0], dev.ordinal, swiglu_bwd_tile_kernel<POW2>, GluBwdSmem::kAlloc);
  if (st != FP8BW_OK) return st;
  const GluTileArgs a{tiles_r, tiles_c, out};
  return launched(launch_kernel(swiglu_bwd_tile_kernel<POW2>, grid, block, GluBwdSmem::kAlloc, cs,
                                mg, mu, md, a));
}

// ---------------------------------------------------------------- Newton-Schulz
constexpr int kMaxSteps = 64;
static_assert(ns::kMaxJobs == FP8BW_NS_MAX_JOBS, "the header's limit");
constexpr int64_t kMaxNsDim = int64_t(1) << 17;

struct NsBuffers {
  uint16_t* hi[2];       // the iterate, alternating
  uint16_t* lo;
  uint16_t* m[3];        // matrices of the short side
  double* part;
};

int64_t ns_align(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Elements per row of a workspace matrix.
int64_t ns_pitch(int64_t cols) { return cdiv(cols, 64) * 64; }

int64_t ns_job_bytes(int64_t n, int64_t k) {
  if (n == 0 || k == 0) return 0;
  const int64_t r = std::min(n, k);
  return 3 * ns_align(2 * n * ns_pitch(k)) + 3 * ns_align(2 * r * ns_pitch(r)) +
         ns_align(8 * ns::kNormBlocks);
}

NsBuffers ns_carve(uint8_t* p, int64_t n, int64_t k) {
  const int64_t r = std::min(n, k);
  const int64_t x = ns_align(2 * n * ns_pitch(k)), m = ns_align(2 * r * ns_pitch(r));
  NsBuffers b;
  b.hi[0] = reinterpret_cast<uint16_t*>(p);
  b.hi[1] = reinterpret_cast<uint16_t*>(p + x);
  b.lo = reinterpret_cast<uint16_t*>(p + 2 * x);
  for (int i = 0; i < 3; ++i) b.m[i] = reinterpret_cast<uint16_t*>(p + 3 * x + i * m);
  b.part = reinterpret_cast<double*>(p + 3 * x + 3 * m);
  return b;
}

bool ns_dims_ok(int64_t n, int64_t k) {
  return n >= 0 && k >= 0 && n % 16 == 0 && k % 16 == 0 && n <= kMaxNsDim && k <= kMaxNsDim;
}

// One GEMM over all jobs: an operand is a workspace matrix with `rows` rows of
// `pitch` elements, read K-major (contraction along the row) or MN-major.
struct NsOperand {
  const uint16_t* p;
  int64_t rows, pitch;
  bool mn;
};
struct NsGemm {
  NsOperand a, b;
  const uint16_t* c;
  const uint16_t* c2;
  uint16_t* out;
  uint16_t* lo;           // not null: the result is an iterate, split into out and lo
  int64_t rows, cols, kc;
  int64_t pitch;          // of c and c2, and of out unless it is the caller's
  bool sym, bf16;
  float alpha, beta, beta2, diag;
};

int64_t ns_tiles(const NsGemm& g, int bn) {
  const int64_t tm = cdiv(g.rows, 256), tn = cdiv(g.cols, bn);
  if (!g.sym) return tm * tn;
  const int64_t per = 256 / bn;
  return tm * tn - per * (tm * (tm - 1) / 2);
}

// The longest cluster's time under the kernel's tile order, in chunks of a
// 256-wide tile. A chunk is weighed by what its two operand boxes cost one SM's TMA
// unit (120 cycles each, and 64 bytes a cycle): 1260 cycles with 256 columns (32 + 32
// KB), 1010 with 128 (32 + 16 KB), 880 with 64 (32 + 8 KB). With all SMs busy a chunk
// takes longer (1980 with 256), about in proportion to its bytes; the weights serve to
// choose a width where few tiles are spread badly. A tile also costs about a chunk of
// pipeline fill.
double ns_makespan(const NsGemm* g, int count, int bn, int clusters) {
  const double chunk = bn == 256 ? 1.0 : bn == 128 ? 0.8 : 0.7;
  int64_t total = 0;
  double sum = 0.0;
  for (int i = 0; i < count; ++i) {
    total += ns_tiles(g[i], bn);
    sum += static_cast<double>(ns_tiles(g[i], bn)) * (cdiv(g[i].kc, ns::BK) + 1) * chunk;
  }
  const int64_t waves = cdiv(total, clusters);
  if (waves > 16) return sum / clusters;      // the last wave hardly counts
  double worst = 0.0;
  for (int c = 0; c < clusters; ++c) {
    double w = 0.0;
    for (int64_t k = 0; k < waves; ++k) {
      int64_t t = k * clusters + ((k & 1) ? clusters - 1 - c : c);
      if (t >= total) continue;
      int i = 0;
      while (t >= ns_tiles(g[i], bn)) t -= ns_tiles(g[i++], bn);
      w += static_cast<double>(cdiv(g[i].kc, ns::BK) + 1) * chunk;
    }
    worst = std::max(worst, w);
  }
  return worst;
}

// 3-D view [column block of 64][row][64] of a workspace matrix; boxes of two
// blocks x `rows` rows (K-major), or of `blocks` blocks x BK rows (MN-major).
int encode_operand(CUtensorMap* map, const NsOperand& o, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  const int st = tensor_map_encoder(&encode);
  if (st != FP8BW_OK) return st;
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(o.rows),
                              static_cast<cuuint64_t>(o.pitch / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * o.pitch), 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(o.mn ? ns::BK : rows),
                             static_cast<cuuint32_t>(o.mn ? rows / 64 : 2)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t*>(o.p), dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? FP8BW_OK
             : FP8BW_ERR_CUDA;
}

template <int BN>
int ns_clusters(const Device& dev, int* clusters) {
  static DevicePrep prep;
  auto kernel = ns::ns_gemm_kernel<BN>;
  return prepare_for_device(prep, dev.ordinal, clusters, [&](int* out) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ns::Layout<BN>::kAlloc) != cudaSuccess)
      return static_cast<int>(FP8BW_ERR_LAUNCH);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * dev.sm_count);
    cfg.blockDim = dim3(ns::kThreads);
    cfg.dynamicSmemBytes = ns::Layout<BN>::kAlloc;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(out, kernel, &cfg) == cudaSuccess && *out >= 1
               ? static_cast<int>(FP8BW_OK)
               : static_cast<int>(FP8BW_ERR_LAUNCH);
  });
}

// One launch over the products g[0 .. count).
int ns_launch(NsGemm* g, int count, const Device& dev, cudaStream_t stream) {
  // long contractions first (see the kernel's tile order)
  std::stable_sort(g, g + count, [](const NsGemm& x, const NsGemm& y) { return x.kc > y.kc; });
  int c256 = 0, c128 = 0, c64 = 0;
  int st = ns_clusters<256>(dev, &c256);
  if (st == FP8BW_OK) st = ns_clusters<128>(dev, &c128);
  if (st == FP8BW_OK) st = ns_clusters<64>(dev, &c64);
  if (st != FP8BW_OK) return st;
  // Narrower tiles where they spread the work better over the clusters (five steps,
  // us, with tiles of 64 and without: 512 x 512 111 and 125, 1024 x 1024 139 and 153,
  // 1024 x 4096 199 and 226)
  int bn = 256, clusters = c256;
  double best = ns_makespan(g, count, 256, c256);
  const double w128 = ns_makespan(g, count, 128, c128);
  if (w128 < 0.97 * best) bn = 128, clusters = c128, best = w128;
  // (64: not with MN-major B, whose 128-byte rows are 64 columns of a CTA)
  bool narrow = true;
  for (int i = 0; i < count; ++i) narrow = narrow && !g[i].b.mn;
  if (narrow && ns_makespan(g, count, 64, c64) < 0.97 * best) bn = 64, clusters = c64;
  ns::Maps maps;
  ns::Args args;
  std::memset(&maps, 0, sizeof maps);
  std::memset(&args, 0, sizeof args);
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i) {
    ns::Job& j = args.job[i];
    j.rows = static_cast<int>(g[i].rows);
    j.cols = static_cast<int>(g[i].cols);
    j.tiles_n = static_cast<int>(cdiv(g[i].cols, bn));
    j.chunks = static_cast<int>(cdiv(g[i].kc, ns::BK));
    tiles += ns_tiles(g[i], bn);
    if (tiles > INT32_MAX / 2) return FP8BW_ERR_SHAPE;
    j.tile_end = static_cast<int>(tiles);
    j.pitch = static_cast<int>(g[i].pitch);
    j.a_mn = g[i].a.mn;
    j.b_mn = g[i].b.mn;
    j.sym = g[i].sym;
    j.split = g[i].lo != nullptr;
    j.bf16 = g[i].bf16;
    j.c = g[i].c;
    j.c2 = g[i].c2;
    j.out = g[i].out;
    j.lo = g[i].lo;
    j.alpha = g[i].alpha;
    j.beta = g[i].beta;
    j.beta2 = g[i].beta2;
    j.diag = g[i].diag;
    st = encode_operand(&maps.a[i], g[i].a, ns::BM);
    if (st == FP8BW_OK) st = encode_operand(&maps.b[i], g[i].b, bn / 2);
    if (st != FP8BW_OK) return st;
  }
  args.count = count;
  const dim3 grid(2 * static_cast<unsigned>(std::min<int64_t>(clusters, tiles))), block(ns::kThreads);
  if (bn == 256)
    return launched(launch_kernel(ns::ns_gemm_kernel<256>, grid, block, ns::Layout<256>::kAlloc,
                                  stream, maps, args));
  if (bn == 128)
    return launched(launch_kernel(ns::ns_gemm_kernel<128>, grid, block, ns::Layout<128>::kAlloc,
                                  stream, maps, args));
  return launched(launch_kernel(ns::ns_gemm_kernel<64>, grid, block, ns::Layout<64>::kAlloc,
                                stream, maps, args));
}

// The products of one matrix's iteration.
struct NsMatrix {
  int64_t n, k, r, c, kp, rp;
  bool tall, pairs;
  NsBuffers w;
  uint16_t* out;
  int parity = 0;
  float ca, cb, cc;

  NsMatrix() = default;
  NsMatrix(const fp8bw_ns_job& j, uint8_t* ws, bool chained, float a, float b, float c_)
      : n(j.n), k(j.k), r(std::min(j.n, j.k)), c(std::max(j.n, j.k)), kp(ns_pitch(j.k)),
        rp(ns_pitch(std::min(j.n, j.k))), tall(j.n > j.k), w(ns_carve(ws, j.n, j.k)),
        out(j.out), ca(a), cb(b), cc(c_) {
    // A pair of steps trades 3 r^2 R flops for 3 r^3 and one launch: for R >= 3/2 r
    // where the products are long beside a launch (2 r^2 R flops of 4 G: 4 us).
    // P_1 P_0 - d_1 d_0 I has to stay below 64, its range at kQScale.
    // In a chain (one launch) the products cost less than the update they save.
    pairs = (chained || (2 * c >= 3 * r && static_cast<double>(r) * r * c >= 2e9)) &&
            std::fabs(ca) <= 5.0f && std::fabs(ca + cb + cc) <= 5.0f;
  }

  // d of P - d I at a step
  float shift(int step) const { return step >= ns::kShiftStep ? ca + cb + cc : ca; }
  NsOperand small(int i) const { return {w.m[i], r, rp, false}; }

  // m[0] = X X^T
  NsGemm gram() const {
    NsGemm g{};
    g.a = g.b = {w.hi[parity], n, kp, tall};
    g.out = w.m[0];
    g.rows = r;
    g.cols = rp;
    g.kc = c;
    g.sym = true;
    g.alpha = ns::kAScale / (ns::kXScale * ns::kXScale);
    return g;
  }
  // m[o] = alpha m[x] m[y] + beta m[p] (symmetric; operands that commute)
  NsGemm product(int o, int x, int y, int p, float alpha, float beta) const {
    NsGemm g{};
    g.a = small(x);
    g.b = small(y);
    g.c = w.m[p];
    g.out = w.m[o];
    g.rows = r;
    g.cols = g.pitch = rp;
    g.kc = r;
    g.sym = true;
    g.alpha = alpha;
    g.beta = beta;
    return g;
  }
  // m[o] = P - d I of A = m[x]
  NsGemm poly(int o, int x, int step) const {
    NsGemm g = product(o, x, x, x, cc / ns::kAScale, cb);
    g.diag = (shift(step) - ca) * ns::kAScale;
    return g;
  }
  // P_1 P_0 - d_1 d_0 I of m[1] and m[2], into m[0]
  NsGemm pair_product(int step) const {
    NsGemm g = product(0, 1, 2, 1, ns::kQScale / (ns::kAScale * ns::kAScale),
                       shift(step + 1) * ns::kQScale / ns::kAScale);
    g.c2 = w.m[2];
    g.beta2 = shift(step) * ns::kQScale / ns::kAScale;
    return g;
  }
  // T = P_0 A_0 and A_1 = T P_0
  NsGemm half_conjugate(int step) const { return product(2, 1, 0, 0, 1.0f / ns::kAScale, shift(step)); }
  NsGemm conjugate(int step) const { return product(0, 2, 1, 2, 1.0f / ns::kAScale, shift(step)); }
  // All of the short side's products of a step (or a pair); the index of the last.
  int short_side(int step, bool pair, NsGemm (&g)[ns::kChainOps]) const {
    g[0] = gram();
    g[1] = poly(1, 0, step);
    if (!pair) return 1;
    g[2] = half_conjugate(step);
    g[3] = conjugate(step);
    g[4] = poly(2, 0, step + 1);
    g[5] = pair_product(step);
    return 5;
  }
  // X <- d X + m[q] X / scale, or the result if `last`
  NsGemm update(int q, float d, float scale, bool last) {
    NsGemm g{};
    const NsOperand x{w.hi[parity], n, kp, !tall};
    g.a = tall ? x : small(q);
    g.b = tall ? small(q) : x;
    g.c = w.hi[parity];
    g.c2 = w.lo;
    g.rows = n;
    g.kc = r;
    g.pitch = kp;
    const float out_scale = last ? 1.0f / ns::kXScale : 1.0f;
    g.alpha = out_scale / scale;
    g.beta = d * out_scale;
    g.beta2 = g.beta / ns::kLoScale;
    g.bf16 = last;
    g.out = last ? out : w.hi[1 - parity];
    g.lo = last ? nullptr : w.lo;
    g.cols = last ? k : kp;
    parity = 1 - parity;
    return g;
  }
};

// One launch: the short sides of all jobs (r <= 256) at a step, up to what multiplies
// X; of the step and the next one, if `pair`.
int ns_chain_launch(const NsMatrix* mat, int count, int step, bool pair, const Device& dev,
                    cudaStream_t stream) {
  ns::ChainMaps maps;
  ns::ChainArgs args;
  std::memset(&maps, 0, sizeof maps);
  std::memset(&args, 0, sizeof args);
  for (int i = 0; i < count; ++i) {
    const NsMatrix& m = mat[i];
    NsGemm g[ns::kChainOps];
    const int last = m.short_side(step, pair, g);
    ns::ChainJob& j = args.job[i];
    j.r = static_cast<int>(m.r);
    j.pitch = static_cast<int>(m.rp);
    j.chunks = static_cast<int>(cdiv(m.c, ns::BK));
    j.last = last;
    j.mn = m.tall;
    j.out = g[last].out;
    for (int k = 0; k <= last; ++k) {
      j.alpha[k] = g[k].alpha;
      j.beta[k] = g[k].beta;
      j.diag[k] = g[k].diag;
    }
    j.beta2 = g[last].beta2;
    const int st = encode_operand(&maps.x[i], g[0].a, ns::BM);
    if (st != FP8BW_OK) return st;
  }
  static DevicePrep prep;
  const int st = allow_smem(prep, dev.ordinal, ns::ns_chain_kernel, ns::ChainLayout::kAlloc);
  if (st != FP8BW_OK) return st;
  return launched(launch_kernel(ns::ns_chain_kernel, dim3(2 * count), dim3(ns::kThreads),
                                ns::ChainLayout::kAlloc, stream, maps, args));
}

int newton_schulz(const fp8bw_ns_job* jobs, int count, int g_is_f32, int steps, float ca, float cb,
                  float cc, float eps, void* ws, int64_t ws_bytes, void* stream) {
  if (count < 0 || count > ns::kMaxJobs || steps < 1 || steps > kMaxSteps || !(eps >= 0.0f) ||
      !std::isfinite(ca) || !std::isfinite(cb) || !std::isfinite(cc))
    return FP8BW_ERR_SHAPE;
  if (count > 0 && jobs == nullptr) return FP8BW_ERR_NULL;
  Buffers b;
  int64_t need = 0;
  for (int i = 0; i < count; ++i) {
    const fp8bw_ns_job& j = jobs[i];
    if (!ns_dims_ok(j.n, j.k)) return FP8BW_ERR_SHAPE;
    b.in(j.g, j.n * j.k * (g_is_f32 ? 4 : 2));
    b.out(j.out, 2 * j.n * j.k);
    need += ns_job_bytes(j.n, j.k);
  }
  if (ws_bytes < need) return FP8BW_ERR_SHAPE;
  b.out(ws, need);
  int st = b.check();
  if (st != FP8BW_OK) return st;
  if (reinterpret_cast<uintptr_t>(ws) % 128 != 0) return FP8BW_ERR_ALIGN;
  Device dev;
  st = current_device(&dev);
  if (st != FP8BW_OK) return st;

  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  NsMatrix mat[ns::kMaxJobs];
  ns::InArgs in{};
  in.g_f32 = g_is_f32 != 0;
  in.eps = eps;
  int nl = 0;
  int64_t most = 0;
  bool any_pairs = false;
  uint8_t* p = static_cast<uint8_t*>(ws);
  // Chains for calls of small matrices only: beside a large one they would be one
  // more launch to wait for, where its launches have room for their tiles.
  bool chained = true;
  for (int i = 0; i < count; ++i)
    chained = chained && std::min(jobs[i].n, jobs[i].k) <= ns::kChainDim;
  for (int i = 0; i < count; ++i) {
    const fp8bw_ns_job& j = jobs[i];
    if (j.n == 0 || j.k == 0) continue;
    mat[nl] = NsMatrix(j, p, chained, ca, cb, cc);
    p += ns_job_bytes(j.n, j.k);
    const NsMatrix& m = mat[nl];
    in.job[nl] = ns::InJob{j.g, j.n * j.k, static_cast<int>(j.k), static_cast<int>(m.kp),
                           m.w.part, m.w.hi[0], m.w.lo};
    most = std::max(most, j.n * m.kp);
    any_pairs = any_pairs || m.pairs;
    ++nl;
  }
  if (nl == 0) return FP8BW_OK;

  st = launched(launch_kernel(ns::ns_sumsq_kernel, dim3(ns::kNormBlocks, nl),
                              dim3(ns::kSplitThreads), 0, cs, in));
  if (st != FP8BW_OK) return st;
  const int64_t blocks = std::min<int64_t>(cdiv(most, 8 * ns::kSplitThreads), 8 * dev.sm_count / nl);
  st = launched(launch_kernel(ns::ns_split_kernel,
                              dim3(static_cast<unsigned>(std::max<int64_t>(1, blocks)), nl),
                              dim3(ns::kSplitThreads), 0, cs, in));

  // One launch: what `make(matrix, &gemm)` gives for every matrix it returns
  // true for.
  auto launch = [&](auto&& make) {
    if (st != FP8BW_OK) return;
    NsGemm g[ns::kMaxJobs];
    int n = 0;
    for (int i = 0; i < nl; ++i)
      if (make(mat[i], &g[n])) ++n;
    if (n > 0) st = ns_launch(g, n, dev, cs);
  };
  const float a = ns::kAScale;
  for (int i = 0; st == FP8BW_OK && i < steps;) {
    // the first two steps and, from five steps on, the last two as a pair
    const bool pair = any_pairs && i + 2 <= steps &&
                      (i == 0 || (steps >= 5 && i == steps - 2));
    const bool last = i + (pair ? 2 : 1) == steps;
    if (chained) {
      st = ns_chain_launch(mat, nl, i, pair, dev, cs);
    } else {
      launch([&](NsMatrix& m, NsGemm* g) { return *g = m.gram(), true; });
      launch([&](NsMatrix& m, NsGemm* g) { return *g = m.poly(1, 0, i), true; });
    }
    if (pair) {
      if (!chained) {
        // matrices that take no pairs go on step by step in the same launches
        launch([&](NsMatrix& m, NsGemm* g) {
          *g = m.pairs ? m.half_conjugate(i) : m.update(1, m.shift(i), a, false);
          return true;
        });
        launch([&](NsMatrix& m, NsGemm* g) {
          return *g = m.pairs ? m.conjugate(i) : m.gram(), true;
        });
        launch([&](NsMatrix& m, NsGemm* g) {
          return *g = m.pairs ? m.poly(2, 0, i + 1) : m.poly(1, 0, i + 1), true;
        });
        launch([&](NsMatrix& m, NsGemm* g) { return *g = m.pair_product(i), m.pairs; });
      }
      launch([&](NsMatrix& m, NsGemm* g) {
        *g = m.pairs ? m.update(0, m.shift(i) * m.shift(i + 1), ns::kQScale, last)
                     : m.update(1, m.shift(i + 1), a, last);
        return true;
      });
    } else {
      launch([&](NsMatrix& m, NsGemm* g) {
        return *g = m.update(1, m.shift(i), a, last), true;
      });
    }
    i += pair ? 2 : 1;
  }
  return st;
}

}  // namespace
}  // namespace layer
}  // namespace fp8bw

using namespace fp8bw;

extern "C" {

int fp8bw_rmsnorm_quantize(const uint16_t* x, const uint16_t* residual, const void* gamma,
                           int gamma_is_f32, int64_t rows, int64_t cols, float eps, uint16_t* h,
                           float* rstd, uint16_t* y, uint8_t* q, float* s, uint8_t* q_t,
                           float* s_t, void* stream) {
  return layer::rmsnorm_quantize<false>(x, residual, gamma, gamma_is_f32, rows, cols, eps, h, rstd,
                                        y, q, s, q_t, s_t, stream);
}

int fp8bw_rmsnorm_quantize_pow2(const uint16_t* x, const uint16_t* residual, const void* gamma,
                                int gamma_is_f32, int64_t rows, int64_t cols, float eps,
                                uint16_t* h, float* rstd, uint16_t* y, uint8_t* q, float* s,
                                uint8_t* q_t, float* s_t, void* stream) {
  return layer::rmsnorm_quantize<true>(x, residual, gamma, gamma_is_f32, rows, cols, eps, h, rstd,
                                       y, q, s, q_t, s_t, stream);
}

int64_t fp8bw_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > layer::kMaxRows || !layer::cols_ok(cols, layer::kMaxNormCols))
    return FP8BW_ERR_SHAPE;
  return rows * cols > 0 ? layer::bwd_plan(rows, cols).blocks * cols * 4 : 0;
}

int fp8bw_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const float* rstd,
                           const void* gamma, int gamma_is_f32, const uint16_t* dres, int64_t rows,
                           int64_t cols, uint16_t* dh, float* dgamma, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  return layer::rmsnorm_backward(dy, h, rstd, gamma, gamma_is_f32, dres, rows, cols, dh, dgamma,
                                 workspace, workspace_bytes, stream);
}

int fp8bw_swiglu_quantize(const uint16_t* gu, int64_t rows, int64_t f, uint8_t* q, float* s,
                          uint8_t* q_t, float* s_t, void* stream) {
  return layer::swiglu_quantize<false>(gu, rows, f, q, s, q_t, s_t, stream);
}

int fp8bw_swiglu_quantize_pow2(const uint16_t* gu, int64_t rows, int64_t f, uint8_t* q, float* s,
                               uint8_t* q_t, float* s_t, void* stream) {
  return layer::swiglu_quantize<true>(gu, rows, f, q, s, q_t, s_t, stream);
}

int fp8bw_swiglu_backward_quantize(const uint16_t* da, const uint16_t* gu, int64_t rows, int64_t f,
                                   uint8_t* q, float* s, uint8_t* q_t, float* s_t, void* stream) {
  return layer::swiglu_backward_quantize<false>(da, gu, rows, f, q, s, q_t, s_t, stream);
}

int fp8bw_swiglu_backward_quantize_pow2(const uint16_t* da, const uint16_t* gu, int64_t rows,
                                        int64_t f, uint8_t* q, float* s, uint8_t* q_t, float* s_t,
                                        void* stream) {
  return layer::swiglu_backward_quantize<true>(da, gu, rows, f, q, s, q_t, s_t, stream);
}

int64_t fp8bw_newton_schulz_workspace(const fp8bw_ns_job* jobs, int count) {
  if (count < 0 || count > ns::kMaxJobs) return FP8BW_ERR_SHAPE;
  if (count > 0 && jobs == nullptr) return FP8BW_ERR_NULL;
  int64_t need = 0;
  for (int i = 0; i < count; ++i) {
    if (!layer::ns_dims_ok(jobs[i].n, jobs[i].k)) return FP8BW_ERR_SHAPE;
    need += layer::ns_job_bytes(jobs[i].n, jobs[i].k);
  }
  return need;
}

int fp8bw_newton_schulz(const fp8bw_ns_job* jobs, int count, int g_is_f32, int steps, float a,
                        float b, float c, float eps, void* workspace, int64_t workspace_bytes,
                        void* stream) {
  return layer::newton_schulz(jobs, count, g_is_f32, steps, a, b, c, eps, workspace,
                              workspace_bytes, stream);
}

int fp8bw_layer_check_device_error(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return FP8BW_ERR_CUDA;
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, fp8bw::g_device_error, sizeof v) != cudaSuccess)
    return FP8BW_ERR_CUDA;
  if (v == 0u) return FP8BW_OK;
  if (cudaMemcpyToSymbol(fp8bw::g_device_error, &zero, sizeof zero) != cudaSuccess)
    return FP8BW_ERR_CUDA;
  return FP8BW_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
