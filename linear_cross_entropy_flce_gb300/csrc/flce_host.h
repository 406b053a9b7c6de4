// Host-side helpers shared by the C-ABI translation units: device query, tensor-map
// encoding, the workspace plan of the GEMM calls and its backward launch sequence.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/flce.h"
#include "flce_internal.h"

namespace flce {

constexpr int64_t kDefaultTimeoutNs = 2000000000LL;
constexpr size_t kGChunkCapBytes = size_t(256) << 20;  // planned bf16 G chunk
constexpr int kMaxDevices = 64;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct DeviceInfo {
  bool init = false;
  int status = FLCE_OK;
  int sms = 0;
};

inline DeviceInfo g_dev[kMaxDevices];
inline std::mutex g_mu;

inline int device_info(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FLCE_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return FLCE_ERR_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.init) {
    int major = 0, minor = 0, count = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      return FLCE_ERR_CUDA;
    }
    d.status = (major == 10 && minor == 3) ? FLCE_OK : FLCE_ERR_DEVICE;
    d.sms = count;
    d.init = true;
  }
  *sms = d.sms;
  return d.status;
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
  });
  return fn;
}

// bf16 matrix [outer][inner] (inner contiguous, row stride ld elements), read in
// boxes of box_inner x box_outer with 128-byte swizzle; out-of-range elements
// read as zero.
inline bool encode_bf16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                 uint32_t box_inner, uint32_t box_outer) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Output map of the GEMM epilogue's TMA stores: [rows][cols] row-major with row
// stride ld elements, boxes of 32 x 32; fp32 boxes use the 128-byte swizzle and
// bf16 boxes the 64-byte one (the layouts the epilogue stages in shared memory).
// Stores outside [rows) x [cols) are dropped, which clips ragged tiles.
inline bool encode_out(CUtensorMap* m, const void* base, bool bf16, uint64_t cols, uint64_t rows,
                uint64_t ld) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const uint64_t esz = bf16 ? 2 : 4;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld * esz};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  bf16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The bf16 G chunk is stored chunk-major, [v_chunk/64][rows][64]: the 64 vocabulary
// ids of one K block of the dH product, or one 64-wide MN chunk of the dW product,
// are contiguous for a run of rows, so each copy of a consumer reads whole
// contiguous blocks (8-16 KB) instead of 128-byte pieces of rows v_chunk·2 bytes
// apart. Three views of it: the gradient epilogue's 32 x 32 store boxes, the
// K-major A operand of dH (64 ids x 128 rows per box) and the MN-major A operand of
// dW (64 ids x 64 rows x 2 chunks per box).
inline bool encode_g_chunked(CUtensorMap* m, void* G, uint64_t rows, uint64_t v_chunk, uint32_t box_x,
                      uint32_t box_y, uint32_t box_z, bool sw64) {
  auto fn = encode_fn();
  if (fn == nullptr || v_chunk % 64 != 0) return false;
  cuuint64_t dims[3] = {64, rows, v_chunk / 64};
  cuuint64_t strides[2] = {128, rows * 128};
  cuuint32_t box[3] = {box_x, box_y, box_z};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, G, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  sw64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  sw64 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Tiles are computed by cluster pairs (tcgen05 cta_group::2, 256-row tiles).
constexpr int kCtaGroup = 2;
// The dW and dH products (K = the token block / the vocabulary chunk, 8192 and
// 16032 at the Llama-3-8B head) run 256 x 512 tiles: a quarter fewer operand bytes
// per flop and fewer distinct operand rows per wave, for an epilogue that no longer
// overlaps the next tile (about 1% of a tile that long). Requested together they
// share one launch, dH's tiles first, because dH alone has too few wide tiles to
// fill the pairs (256 for 76 pairs at the Llama-3-8B head: a last wave 37% full);
// dH alone keeps 256 x 256 tiles.
constexpr bool kWideDw = true;
constexpr bool kWideDhAlone = false;

// MN-major bf16 operand [rows][mn] (mn contiguous, mn % 64 == 0, row stride ld
// elements) as a 3-D map [mn/64][rows][64] read in boxes of 64 x box_rows x
// box_chunks with 128-byte swizzle. The view covers exactly the 2-D tensor, so
// every address it can form lies inside it; rows past the end read as zero.
inline bool encode_bf16_mn3(CUtensorMap* m, const void* base, uint64_t mn, uint64_t rows, uint64_t ld,
                     uint32_t box_rows, uint32_t box_chunks) {
  auto fn = encode_fn();
  if (fn == nullptr || mn % 64 != 0) return false;
  cuuint64_t dims[3] = {64, rows, mn / 64};
  cuuint64_t strides[2] = {ld * 2, 128};
  cuuint32_t box[3] = {64, box_rows, box_chunks};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

struct Plan {
  int64_t N = 0, D = 0, V = 0;
  int cta = kCtaGroup;  // CTAs per tile
  int tile_m = BM * kCtaGroup;
  int m_blocks = 0;     // ceil(N / tile_m): row tiles of the forward pass
  int part_stride = 0;  // 128-row blocks per vocabulary range in the partials
  int v_tiles = 0;    // ceil(V / BN)
  int splits = 0;     // forward vocabulary ranges per token block
  int64_t n_block = 0, v_chunk = 0;
  int n_nblocks = 0, n_chunks = 0;
  bool need_dh_acc = false, need_dw_acc = false;
  size_t off_part = 0, off_zt = 0, off_nll = 0, off_lse = 0, off_scal = 0, off_gstat = 0,
         off_g = 0, off_dhacc = 0, off_dwacc = 0, total = 0;
};

inline int choose_splits(int m_blocks, int v_tiles, int sms) {
  // Minimise (waves of units) x (tiles per unit); ties go to fewer splits.
  int best = 1;
  int64_t best_cost = INT64_MAX;
  const int max_s = std::min(v_tiles, 128);
  for (int s = 1; s <= max_s; ++s) {
    const int64_t waves = ceil_div(static_cast<int64_t>(m_blocks) * s, sms);
    const int64_t cost = waves * ceil_div(v_tiles, s);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// backward = false: only the forward pieces (partials, target logits, NLL, lse,
// scalars); the G chunk and the dH / dW accumulators are left out of the total.
inline int make_plan(int64_t N, int64_t D, int64_t V, const flce_options& o, int sms, Plan* P,
              bool backward = true) {
  Plan p;
  p.N = N;
  p.D = D;
  p.V = V;
  p.m_blocks = static_cast<int>(ceil_div(N, p.tile_m));
  p.part_stride = p.m_blocks * p.cta;
  p.v_tiles = static_cast<int>(ceil_div(V, BN));
  if (o.v_splits < 0 || o.v_splits > p.v_tiles) return FLCE_ERR_OPTION;
  p.splits = o.v_splits > 0 ? o.v_splits
                            : choose_splits(p.m_blocks, p.v_tiles, std::max(1, sms / p.cta));

  const int64_t v_round = ceil_div(V, BN) * BN;
  if (o.v_chunk < 0 || o.n_block < 0) return FLCE_ERR_OPTION;
  if (o.v_chunk > 0 && o.v_chunk % BN != 0) return FLCE_ERR_OPTION;
  if (o.n_block > 0 && o.n_block % BM != 0) return FLCE_ERR_OPTION;
  // Planned G chunk: vocabulary chunks of at most 16384 ids, balanced in length
  // (a chunk's dH accumulation and launch ramp are paid per chunk, so fewer,
  // longer chunks are faster); the tokens form one block unless one chunk of G
  // would exceed kGChunkCapBytes, in which case they are split into equal
  // blocks of whole 256-row pair tiles. Measured on GB300: long-sequence head
  // 99.7 -> 93.9 ms with half the workspace, Llama-2-like head 1.93 -> 1.40 ms.
  int64_t cv = o.v_chunk, nb = o.n_block;
  if (cv == 0) {
    const int64_t chunks = ceil_div(V, 16384);
    cv = ceil_div(ceil_div(V, chunks), BN) * BN;
  }
  if (nb == 0) {
    const int64_t bytes = ceil_div(N, BM * 2) * (BM * 2) * cv * 2;
    const int64_t blocks = std::max<int64_t>(1, ceil_div(bytes, static_cast<int64_t>(kGChunkCapBytes)));
    nb = blocks == 1 ? N : ceil_div(ceil_div(N, blocks), BM * 2) * (BM * 2);
  }
  cv = std::min(cv, v_round);
  nb = std::min(nb, N);
  p.v_chunk = cv;
  p.n_block = nb;
  p.n_chunks = static_cast<int>(ceil_div(V, cv));
  p.n_nblocks = static_cast<int>(ceil_div(N, nb));
  p.need_dh_acc = p.n_chunks > 1;
  p.need_dw_acc = (o.dw_dtype == FLCE_DTYPE_BF16) && p.n_nblocks > 1;

  const int64_t rows_b = ceil_div(nb, p.tile_m) * p.tile_m;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  p.off_part = take(static_cast<size_t>(p.splits) * p.part_stride * BM * sizeof(float2));
  p.off_zt = take(static_cast<size_t>(N) * 4);
  p.off_nll = take(static_cast<size_t>(N) * 4);
  p.off_lse = take(static_cast<size_t>(N) * 4);
  p.off_scal = take(256);
  if (backward) {
    p.off_gstat = take(static_cast<size_t>(N) * 16);   // float4 per token
    p.off_g = take(static_cast<size_t>(rows_b) * cv * 2);
    p.off_dhacc = p.need_dh_acc ? take(static_cast<size_t>(rows_b) * D * 4) : off;
    p.off_dwacc = p.need_dw_acc ? take(static_cast<size_t>(V) * D * 4) : off;
  } else {
    p.off_gstat = p.off_g = p.off_dhacc = p.off_dwacc = off;
  }
  p.total = off;
  *P = p;
  return FLCE_OK;
}

inline int check_options(const flce_options& o) {
  if (o.reduction != FLCE_REDUCTION_MEAN && o.reduction != FLCE_REDUCTION_SUM &&
      o.reduction != FLCE_REDUCTION_NONE)
    return FLCE_ERR_OPTION;
  if (o.dw_dtype != FLCE_DTYPE_F32 && o.dw_dtype != FLCE_DTYPE_BF16) return FLCE_ERR_OPTION;
  if (!(o.normalizer >= 0.f) || !(o.grad_scale == o.grad_scale)) return FLCE_ERR_OPTION;
  if (o.timeout_ns < 0) return FLCE_ERR_OPTION;
  if (o.trace_capacity < 0 || (o.trace_capacity > 0 && o.trace_events == nullptr) ||
      o.reserved != 0)
    return FLCE_ERR_OPTION;
  return FLCE_OK;
}

inline int check_shape(int64_t N, int64_t D, int64_t V) {
  if (N < 1 || D < 1 || V < 1) return FLCE_ERR_SHAPE;
  // int32 coordinates and indices inside the kernels
  if (N > (int64_t(1) << 30) || V > (int64_t(1) << 30) || D > (int64_t(1) << 20))
    return FLCE_ERR_SHAPE;
  if (D % 8 != 0) return FLCE_ERR_ALIGN;
  return FLCE_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// uint8 matrix [outer][inner] read in boxes of box_inner x box_outer bytes with
// 128-byte swizzle; out-of-range elements read as zero.
inline bool encode_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
               uint32_t box_inner, uint32_t box_outer) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}


// Optional per-kernel trace of a call: event 0 before its first kernel, event k
// after its k-th.
struct KernelTrace {
  void* const* events = nullptr;
  int capacity = 0;
  cudaStream_t stream = nullptr;
  int n = 0;
  bool operator()() {
    if (events == nullptr || n >= capacity) return true;
    const bool ok = cudaEventRecord(static_cast<cudaEvent_t>(events[n]), stream) == cudaSuccess;
    ++n;
    return ok;
  }
};

// What launch_backward_products needs besides the plan.
struct BackwardProducts {
  const uint16_t* H = nullptr;  // bf16 operands of dW = G^T H and dH = G W
  const uint16_t* W = nullptr;
  const CUtensorMap* h_k = nullptr;  // operands of the recomputed logits
  const CUtensorMap* w_k = nullptr;
  // the gradient GEMM's launcher and the parameters that do not change from chunk to chunk
  cudaError_t (*launch_grad)(int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                             const GemmParams&, int, cudaStream_t, int) = nullptr;
  int fp8 = 0;
  GemmParams grad{};
  int64_t v_base = 0;           // vocabulary id of W's row 0
  uint16_t* dH = nullptr;       // bf16 dH, or
  float* dh_f32 = nullptr;      // the fp32 dH part of a vocabulary shard
  void* dW = nullptr;
  bool dw_bf16 = false;
  uint16_t* G = nullptr;        // workspace: the chunk of G and the accumulators
  float* dh_acc = nullptr;
  float* dw_acc = nullptr;
  int64_t timeout_ns = 0;
  int32_t* status = nullptr;
  int sms = 0;
  cudaStream_t stream = nullptr;
};
int launch_backward_products(const Plan& P, const BackwardProducts& b, KernelTrace& trace);

}  // namespace flce
