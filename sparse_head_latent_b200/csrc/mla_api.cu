// mla_api.cu -- host side of the C ABI declared in include/mla.h:
// argument validation, workspace carving, TMA tensor-map encoding, launch
// sequencing on the caller's stream, device error word and per-kernel
// event timing. All kernels live in the headers included below (one
// translation unit, so no relocatable device code is needed).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/mla.h"
#include "attn.cuh"
#include "attn_abs.cuh"
#include "attn_tree.cuh"
#include "dequant.cuh"
#include "gemm2.cuh"
#include "gemm_w8t.cuh"
#include "gemm8.cuh"
#include "gemm_m64.cuh"
#include "gemm_m64_w8.cuh"
#include "pages.cuh"
#include "prepass.cuh"
#include "quant.cuh"
#include "ptx.cuh"
#include "rope.cuh"

// Device error word: kernels record the first error code here.
__device__ int g_mla_device_error;

namespace {

constexpr int kDn = 128, kDr = 64, kDv = 128, kL = 512, kD = 7168;
using Gemm2Kvb = mla::Gemm2Cfg<false>;  // latent x W_kvb^T  (B stored [N, K])
using Gemm2KvbAttn = mla::Gemm2Cfg<false, true>;  // same, v columns written as f16 for the attention
using Gemm2Wo = mla::Gemm2Cfg<true>;    // attn x W_o         (B stored [K, N]); also q_nope x W_UK
using Gemm2Unabs = mla::Gemm2Cfg<false, false, 128>;  // o_lat x W_UV^T (B stored [N, K], 128 wide)
using Gemm2WoNarrow = mla::Gemm2Cfg<true, false, 128>;
using GemmW8tKvb = mla::GemmW8tCfg<false, true>;            // latent x e4m3 W_kvb^T, weights converted on chip
using GemmW8tKvbAttn = mla::GemmW8tCfg<false, true, true>;  // same, v columns written as f16 for the attention
using GemmW8tWo = mla::GemmW8tCfg<true, false>;             // attn x e4m3 W_o, weights converted on chip  // attn x W_o with one row tile (decode): twice the pairs
using GemmM64 = mla::GemmM64Cfg<64>;     // decode's output projection (stream-K), M <= 64
using GemmM128 = mla::GemmM64Cfg<128>;   // and 64 < M <= 256 (128-row tiles)
using GemmM64Abs = mla::GemmM64Cfg<64, true, true>;     // decode's q_nope x W_UK per head, bf16 out
using GemmM128Abs = mla::GemmM64Cfg<128, true, true>;
using GemmM64Unabs = mla::GemmM64Cfg<64, false, true>;  // decode's o_lat x W_UV^T per head, bf16 out
using GemmM128Unabs = mla::GemmM64Cfg<128, false, true>;
using GemmW8Wo64 = mla::GemmM64W8Cfg<64, true, false>;      // the same three over e4m3 codes (tree decode)
using GemmW8Wo128 = mla::GemmM64W8Cfg<128, true, false>;
using GemmW8Abs64 = mla::GemmM64W8Cfg<64, true, true>;
using GemmW8Abs128 = mla::GemmM64W8Cfg<128, true, true>;
using GemmW8Unabs64 = mla::GemmM64W8Cfg<64, false, true>;
using GemmW8Unabs128 = mla::GemmM64W8Cfg<128, false, true>;
using Gemm8Kvb = mla::Gemm8Cfg<false>;              // e4m3 latent x e4m3 W_kvb^T
using Gemm8KvbAttn = mla::Gemm8Cfg<false, true>;    // same, v tiles written as f16 for the attention
using Gemm8Wo = mla::Gemm8Cfg<true>;           // e4m3 attn x e4m3 W_o (B stored [K, N])

// ------------------------------------------------------------------ device state

struct DeviceState {
  bool ready = false;
  int status = MLA_OK;
  int sms = 0;
  int pairs_kvb = 0;   // CTA pairs of the pair GEMMs that fit on the device at once
  int pairs_wo = 0;
  int pairs_w8t_kvb = 0;  // CTA pairs of the e4m3-weight GEMMs with on-chip conversion
  int pairs_w8t_wo = 0;
  int pairs_unabs = 0;
  int pairs_wo_narrow = 0;
  int pairs8_kvb = 0;  // CTA pairs of the e4m3 GEMMs
  int pairs8_wo = 0;
  int pairs_tree = 0;  // CTA pairs of the tree attention
  int* err = nullptr;  // address of g_mla_device_error on this device
};

template <class Kernel>
int max_pairs(Kernel k, int smem, int threads = 192) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) return 0;
  return n;
}

std::mutex g_mutex;
std::vector<DeviceState> g_devices;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

// One-time set-up per device: device checks, kernel attributes, address of
// the error word. Returns an mla_status.
int device_state(DeviceState** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (static_cast<int>(g_devices.size()) <= dev) g_devices.resize(dev + 1);
  DeviceState& st = g_devices[dev];
  if (!st.ready) {
    st.ready = true;
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) {
      st.status = MLA_ERR_CUDA;
    } else if (prop.major != 10) {
      st.status = MLA_ERR_UNSUPPORTED;  // built for sm_100a only
    } else {
      st.sms = prop.multiProcessorCount;
      bool ok = cudaGetSymbolAddress(reinterpret_cast<void**>(&st.err), g_mla_device_error) == cudaSuccess;
      ok = ok && cudaMemset(st.err, 0, sizeof(int)) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_tc2_kernel<Gemm2Kvb>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      Gemm2Kvb::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_tc2_kernel<Gemm2Wo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      Gemm2Wo::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_tc2_kernel<Gemm2KvbAttn>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, Gemm2KvbAttn::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_tc2_kernel<Gemm2Unabs>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, Gemm2Unabs::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_tc2_kernel<Gemm2WoNarrow>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, Gemm2WoNarrow::SMEM_BYTES) == cudaSuccess;
      if (ok) {
        st.pairs_kvb = max_pairs(mla::gemm_bf16_tc2_kernel<Gemm2Kvb>, Gemm2Kvb::SMEM_BYTES);
        st.pairs_wo = max_pairs(mla::gemm_bf16_tc2_kernel<Gemm2Wo>, Gemm2Wo::SMEM_BYTES);
        ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_w8t_kernel<GemmW8tKvb>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, GemmW8tKvb::SMEM_BYTES) == cudaSuccess;
        ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_w8t_kernel<GemmW8tKvbAttn>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, GemmW8tKvbAttn::SMEM_BYTES) == cudaSuccess;
        ok = ok && cudaFuncSetAttribute(mla::gemm_bf16_w8t_kernel<GemmW8tWo>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, GemmW8tWo::SMEM_BYTES) == cudaSuccess;
        st.pairs_w8t_kvb = max_pairs(mla::gemm_bf16_w8t_kernel<GemmW8tKvb>, GemmW8tKvb::SMEM_BYTES, GemmW8tKvb::THREADS);
        st.pairs_w8t_wo = max_pairs(mla::gemm_bf16_w8t_kernel<GemmW8tWo>, GemmW8tWo::SMEM_BYTES, GemmW8tWo::THREADS);
        st.pairs_unabs = max_pairs(mla::gemm_bf16_tc2_kernel<Gemm2Unabs>, Gemm2Unabs::SMEM_BYTES);
        st.pairs_wo_narrow = max_pairs(mla::gemm_bf16_tc2_kernel<Gemm2WoNarrow>, Gemm2WoNarrow::SMEM_BYTES);
        ok = ok && st.pairs_kvb > 0 && st.pairs_wo > 0 && st.pairs_w8t_kvb > 0 && st.pairs_w8t_wo > 0 && st.pairs_unabs > 0 && st.pairs_wo_narrow > 0;
      }
      ok = ok && cudaFuncSetAttribute(mla::gemm_e4m3_tc2_kernel<Gemm8Kvb>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      Gemm8Kvb::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_e4m3_tc2_kernel<Gemm8KvbAttn>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, Gemm8KvbAttn::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_e4m3_tc2_kernel<Gemm8Wo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      Gemm8Wo::SMEM_BYTES) == cudaSuccess;
      if (ok) {
        st.pairs8_kvb = max_pairs(mla::gemm_e4m3_tc2_kernel<Gemm8Kvb>, Gemm8Kvb::SMEM_BYTES, Gemm8Kvb::THREADS);
        st.pairs8_wo = max_pairs(mla::gemm_e4m3_tc2_kernel<Gemm8Wo>, Gemm8Wo::SMEM_BYTES, Gemm8Wo::THREADS);
        ok = st.pairs8_kvb > 0 && st.pairs8_wo > 0;
      }
      ok = ok && cudaFuncSetAttribute(mla::gemm_m64_kernel<GemmM64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      GemmM64::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_m64_kernel<GemmM128>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, GemmM128::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_m64_kernel<GemmM64Abs>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, GemmM64Abs::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_m64_kernel<GemmM128Abs>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, GemmM128Abs::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_m64_kernel<GemmM64Unabs>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, GemmM64Unabs::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::gemm_m64_kernel<GemmM128Unabs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      GemmM128Unabs::SMEM_BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::absorbed_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      mla::AbsSmem::BYTES) == cudaSuccess;
      auto w8_smem = [](auto kernel, int bytes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
      };
      ok = ok && w8_smem(mla::gemm_m64_w8_kernel<GemmW8Wo64>, GemmW8Wo64::SMEM_BYTES) &&
           w8_smem(mla::gemm_m64_w8_kernel<GemmW8Wo128>, GemmW8Wo128::SMEM_BYTES) &&
           w8_smem(mla::gemm_m64_w8_kernel<GemmW8Abs64>, GemmW8Abs64::SMEM_BYTES) &&
           w8_smem(mla::gemm_m64_w8_kernel<GemmW8Abs128>, GemmW8Abs128::SMEM_BYTES) &&
           w8_smem(mla::gemm_m64_w8_kernel<GemmW8Unabs64>, GemmW8Unabs64::SMEM_BYTES) &&
           w8_smem(mla::gemm_m64_w8_kernel<GemmW8Unabs128>, GemmW8Unabs128::SMEM_BYTES);
      ok = ok && cudaFuncSetAttribute(mla::tree_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      mla::TreeSmem::BYTES) == cudaSuccess;
      if (ok) {
        st.pairs_tree = max_pairs(mla::tree_attn_kernel, mla::TreeSmem::BYTES, mla::kTreeThreads);
        if (st.pairs_tree > mla::kTreeMaxPairs) st.pairs_tree = mla::kTreeMaxPairs;
        ok = st.pairs_tree > 0;
      }
      ok = ok && cudaFuncSetAttribute(mla::sparse_mla_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      mla::AttnSmem::BYTES) == cudaSuccess;
      ok = ok && cudaFuncSetAttribute(mla::topk_bitmap_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      mla::kPrepassWarps * (MLA_MAX_T / 128) * 16) == cudaSuccess;
      if (ok && g_encode == nullptr) {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
             q == cudaDriverEntryPointSuccess && fn != nullptr;
        if (ok) g_encode = reinterpret_cast<EncodeTiledFn>(fn);
      }
      st.status = ok ? MLA_OK : MLA_ERR_CUDA;
    }
  }
  *out = &st;
  return st.status;
}

// ------------------------------------------------------------------ tensor maps

// Row-major bf16/u8 matrix [outer, inner] with a row pitch; box
// [box_outer, box_inner]; 128-byte swizzle; out-of-range rows read as zero.
bool map_2d(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t inner, uint64_t outer,
            uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_outer,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {pitch_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t es[2] = {1, 1};
  return g_encode(m, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 tensor [B, T, inner] (row pitch inner*2 bytes), box [1, box_rows, 64];
// rows past T read as zero.
bool map_3d_bt(CUtensorMap* m, const void* base, uint64_t inner, uint64_t T, uint64_t B, uint32_t box_rows = 128) {
  const cuuint64_t dims[3] = {inner, T, B};
  const cuuint64_t strides[2] = {inner * 2, inner * 2 * T};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 matrix [rows, 512] as 64-column chunks, [rows][8][64]: a box is
// box_chunks chunks of box_rows rows, each chunk contiguous in shared memory;
// rows past the last read as zero.
bool map_chunks(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows, uint32_t box_chunks) {
  const cuuint64_t dims[3] = {64, rows, 8};
  const cuuint64_t strides[2] = {1024, 128};
  const cuuint32_t box[3] = {64, box_rows, box_chunks};
  const cuuint32_t es[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Test hook (mla_test_withhold_attention_loads): whose loads stop early.
enum Withhold : int {
  kWithholdNone = 0,
  kWithholdDense = 1,    // block-dense attention: all of them (a device variable, too)
  kWithholdTree = 2,     // tree attention: keys after a tile's first block
  kWithholdFewRows = 3,  // few-row GEMMs: activations after a CTA's first tile
};
int g_withhold = kWithholdNone;

// How e4m3 weights meet bf16 activations (mla_set_e4m3_weight_conversion):
// 0 = dequantised into a bf16 workspace copy per call, 1 = converted on chip
// by the projection GEMMs.
int g_e4m3_onchip = 0;

// ------------------------------------------------------------------ profiling

struct ProfRecord {
  int cls;
  cudaEvent_t start, stop;
};

struct Profiler {
  bool on = false;
  std::vector<ProfRecord> recs;
  std::vector<cudaEvent_t> pool;
  cudaEvent_t get() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    cudaEventCreate(&e);
    return e;
  }
};
thread_local Profiler t_prof;

// Runs `launch` on `stream`, bracketed by events when profiling is on.
template <class F>
int timed_launch(int cls, cudaStream_t stream, F&& launch) {
  ProfRecord r{cls, nullptr, nullptr};
  if (t_prof.on) {
    r.start = t_prof.get();
    r.stop = t_prof.get();
    cudaEventRecord(r.start, stream);
  }
  launch();
  const cudaError_t e = cudaGetLastError();
  if (t_prof.on) {
    cudaEventRecord(r.stop, stream);
    t_prof.recs.push_back(r);
  }
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

// Launch of a kernel on `st`, as a dependent of the one before it if asked for
// (see griddep_wait): then that one must call griddep_launch, the kernel must
// call griddep_wait before it touches anything the chain's kernels write, and the
// chain must begin with a plain launch. What the chain writes changes while a
// dependent kernel runs, so the kernel takes it without const __restrict__ and
// reads it without __ldg: both say that it never does, and would allow the reads
// to be moved in front of griddep_wait.
template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                          bool dependent, unsigned cluster, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (dependent) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace

// ------------------------------------------------------------------ validation and workspace

namespace {

constexpr size_t kNone = ~size_t(0);
constexpr int64_t kMaxRows = int64_t(1) << 24;  // B*T limit (int32 tile coordinates with margin)

struct WsLayout {
  size_t kvh = kNone, attn = kNone, bitmap = kNone, blocks = kNone, wkvb = kNone, wo = kNone;
  size_t qabs = kNone, olat = kNone, lists = kNone, counts = kNone;  // absorbed path, one chunk of rows
  size_t part_ml = kNone, part_o = kNone;  // decode: partial results of split rows
  size_t lat8 = kNone, lat8_s = kNone;    // e4m3 activations: quantized latent and its scales
  size_t attn8 = kNone, attn8_s = kNone;  // e4m3 activations: quantized attention rows and scales
  int parts = 1;                          // decode: CTAs per (sequence, 64-head group)
  size_t wo_part = kNone;                 // decode: stream-K partial tiles of the output projection
  size_t tree_start = kNone, tree_ml = kNone, tree_o = kNone;  // tree decode: unit starts, partial tiles
  size_t wo_split = kNone;                // prefill: partial tiles of the output projection's K-split last wave
  int g_abs = 0;       // first tile group on the absorbed path (groups of 4 x 128 query rows)
  int abs_chunk = 0;   // absorbed rows processed per pass
  int kpad = 0;        // pitch of the per-row key lists
  size_t total = 0;
};

// Absorbed rows are processed in passes of at most this many rows of one
// batch element, which bounds the workspace (q_abs and o_lat are
// rows x H x 1 KB each).
constexpr int kAbsChunkRows = 2048;
// SM count the decode split is planned for (the workspace size cannot depend
// on the device; a different count only changes how full the waves are).
constexpr int kSmsForSplit = 148;
constexpr int kStreamKCtas = 256;  // upper bound on the stream-K grid (the SM count)
static_assert(kStreamKCtas <= mla::kSumThreads, "a thread of the sum looks at one CTA");
// K-split last wave of the prefill output projection (wo_split_plan): only
// for K of at least kSplitMinTileKb 64-deep blocks (H >= 32; a shorter tile's
// last wave ends before the partial sums would pay), each K range keeps at
// least kSplitMinKb blocks, and the workspace holds kSplitSlots partial tiles
// (the pair count of a 148-SM part; with more pairs the split only gets
// coarser).
constexpr int kSplitMinTileKb = 64;
constexpr int kSplitMinKb = 8;
constexpr int kSplitSlots = 74;
// Up to this many rows the per-head GEMMs run on the few-row kernel (64- or
// 128-row UMMA tiles, one CTA per item), beyond it on the CTA-pair GEMM.
constexpr int kFewRows = 256;
// Trees over e4m3 codes: read as stored up to this many rows (each 128 rows
// convert them again), through bf16 copies (95 us of 128 heads, once) and the
// CTA-pair GEMM, whose last wave is not split along K here, beyond. Whole steps of 4
// nodes over 200 positions, us, codes / copies:
//   heads  256 rows       384            512            768            1024
//   8      46.1 / 48.3    60.6 / 59.0    66.8 / 61.2    86.2 / 78.4    103 / 89
//   16     52.4 / 61.2    70.8 / 74.8    79.9 / 78.0    103 / 100      125 / 110
//   64     94.0 / 143     132 / 160      162 / 171      235 / 241      315 / 277
//   128    157 / 254      231 / 290      304 / 321      466 / 486      595 / 537
// One number for all of them: with 8 heads 384 would be right, and 768 costs 10 %.
constexpr int kFewRowsE4m3 = 768;
// Over bf16 weights: the few-row kernels, launched as dependents, against W_o on the
// pair GEMM in plain launches. The same steps:
//   heads  64 rows        128            192            256
//   8      37.5 / 40.5    39.2 / 38.1    40.1 / 39.5    44.2 / 40.3
//   16     40.8 / 46.9    43.8 / 45.3    47.4 / 45.5    50.0 / 47.1
//   64     61.8 / 78.2    68.7 / 81.7    92.2 / 93.4    96.7 / 96.7
//   128    84.4 / 121     103 / 135      155 / 153      173 / 172
constexpr int kFewRowsTree = 192;
constexpr int64_t tree_few_rows(bool e4m3) { return e4m3 ? kFewRowsE4m3 : kFewRowsTree; }
// Cost model for MLA_PATH_AUTO: a tile group goes absorbed when its middle
// row's causal prefix exceeds this many times the selection size. Measured
// on B200 at T = 32768, H = 128, top-k 2048: the block-dense kernel costs
// about 80 ps per (row, prefix key) for all heads, the absorbed kernel about
// 870 ps per (row, selected key) (2176 instead of 640 FLOP per head and key,
// M = 64 UMMAs, and every 64-head group gathers the row's keys from L2).
constexpr int kAbsorbRatio = 11;

// First tile group that runs on the absorbed path (== number of groups when
// none does).
int absorbed_first_group(const mla_dims& d, bool has_topk) {
  const int nq = (d.T + 127) / 128;
  const int ng = (nq + 3) / 4;
  if (!has_topk || d.path == MLA_PATH_BLOCK_DENSE || d.act == MLA_ACT_E4M3_DYNAMIC) return ng;
  if (d.path == MLA_PATH_ABSORBED) return 0;
  const int64_t k = d.topk < d.T ? d.topk : d.T;
  for (int g = 0; g < ng; ++g)
    if (int64_t(512) * g + 256 > int64_t(kAbsorbRatio) * k) return g;
  return ng;
}

int check_dims(const mla_dims* d) {
  if (d == nullptr) return MLA_ERR_NULL;
  if (d->d_nope != kDn || d->d_rope != kDr || d->d_v != kDv || d->d_latent != kL || d->d_model != kD)
    return MLA_ERR_UNSUPPORTED;
  if (d->wdtype != MLA_W_BF16 && d->wdtype != MLA_W_E4M3_BLOCK128) return MLA_ERR_UNSUPPORTED;
  if (d->B < 0 || d->T < 0 || d->H < 1 || d->T > MLA_MAX_T) return MLA_ERR_SHAPE;
  if (static_cast<int64_t>(d->B) * d->T > kMaxRows) return MLA_ERR_SHAPE;
  if (d->path != MLA_PATH_AUTO && d->path != MLA_PATH_BLOCK_DENSE && d->path != MLA_PATH_ABSORBED)
    return MLA_ERR_UNSUPPORTED;
  if (d->act != MLA_ACT_BF16 && d->act != MLA_ACT_E4M3_DYNAMIC) return MLA_ERR_UNSUPPORTED;
  if (d->act == MLA_ACT_E4M3_DYNAMIC && (d->wdtype != MLA_W_E4M3_BLOCK128 || d->path == MLA_PATH_ABSORBED))
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

WsLayout ws_layout(const mla_dims& d, int entry, bool has_topk) {
  WsLayout w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) & ~size_t(255);
    return o;
  };
  const size_t rows = static_cast<size_t>(d.B) * d.T;
  const size_t H = d.H;
  const size_t nq = (static_cast<size_t>(d.T) + 127) / 128;
  const bool fp8 = d.wdtype == MLA_W_E4M3_BLOCK128;
  const bool attend = entry == MLA_ENTRY_ATTEND || entry == MLA_ENTRY_PREFILL;
  if (attend) {
    w.g_abs = absorbed_first_group(d, has_topk);
    if (w.g_abs > 0) w.kvh = take(rows * H * (kDn + kDv) * 2);  // block-dense rows only
    // The whole block keeps the attention rows in the workspace (as e4m3
    // codes + scales when the activations are quantized, see below).
    if (entry == MLA_ENTRY_PREFILL && d.act != MLA_ACT_E4M3_DYNAMIC) w.attn = take(rows * H * kDv * 2);
    if (has_topk) {
      w.bitmap = take(static_cast<size_t>(d.B) * (nq * (nq + 1) / 2) * 128 * 16);
      w.blocks = take(static_cast<size_t>(d.B) * ((nq + 3) / 4) * (nq + 2) * 4);
    }
    const int64_t abs_rows = int64_t(d.T) - int64_t(512) * w.g_abs;
    if (abs_rows > 0 && d.B > 0) {
      w.abs_chunk = static_cast<int>(abs_rows < kAbsChunkRows ? abs_rows : kAbsChunkRows);
      const int k = d.topk < d.T ? d.topk : d.T;
      w.kpad = (k + 63) / 64 * 64;
      const size_t ch = static_cast<size_t>(w.abs_chunk);
      w.qabs = take(ch * H * kL * 2);
      w.olat = take(ch * H * kL * 2);
      w.lists = take(ch * static_cast<size_t>(w.kpad) * 4);
      w.counts = take(ch * 4);
    }
  }
  if (entry == MLA_ENTRY_DECODE && d.B > 0) {
    const size_t B = d.B;
    const int k = has_topk ? (d.topk < d.T ? d.topk : d.T) : d.T;
    w.kpad = (k + 63) / 64 * 64;
    w.qabs = take(B * H * kL * 2);
    w.olat = take(B * H * kL * 2);
    w.lists = take(B * static_cast<size_t>(w.kpad) * 4);
    w.counts = take(B * 4);
    w.attn = take(B * H * kDv * 2);
    // Split each sequence's keys over several CTAs when B alone cannot fill
    // the device: about two waves of CTAs, at least four 64-key blocks each.
    const int hgroups = (d.H + 63) / 64;
    const int want = (2 * kSmsForSplit + d.B * hgroups - 1) / (d.B * hgroups);
    const int most = w.kpad / 64 / 4;
    w.parts = want < most ? want : most;
    if (w.parts > 16) w.parts = 16;
    if (w.parts < 1) w.parts = 1;
    if (w.parts > 1) {
      w.part_ml = take(B * w.parts * H * 8);
      w.part_o = take(B * w.parts * H * kL * 2);
    }
    // The output projection of up to 256 rows runs as a stream-K GEMM with
    // 64- or 128-row tiles: one fp32 partial tile per (CTA, tile) segment.
    if (d.B <= 256) {
      const int bm = d.B <= 64 ? 64 : 128;
      const size_t tiles = static_cast<size_t>((d.B + bm - 1) / bm) * (kD / 128);
      w.wo_part = take((kStreamKCtas + tiles) * bm * 128 * 4);
    }
  }
  if (entry == MLA_ENTRY_TREE_DECODE && rows > 0) {
    w.qabs = take(rows * H * kL * 2);
    w.olat = take(rows * H * kL * 2);
    w.attn = take(rows * H * kDv * 2);
    w.tree_start = take((static_cast<size_t>(d.B) + 2) * 8);
    w.tree_ml = take(size_t(2) * mla::kTreeMaxPairs * mla::kTreeRows * 8);
    w.tree_o = take(size_t(2) * mla::kTreeMaxPairs * mla::kTreeSlotFloats * 4);
    if (rows <= tree_few_rows(fp8)) {
      const int bm = rows <= 64 ? 64 : 128;
      const size_t tiles = (rows + bm - 1) / bm * (kD / 128);
      w.wo_part = take((kStreamKCtas + tiles) * bm * 128 * 4);
    }
  }
  // Decoding reads bf16 copies of e4m3 weights; trees of few rows the codes.
  const bool copies = entry == MLA_ENTRY_DECODE || (entry == MLA_ENTRY_TREE_DECODE && rows > kFewRowsE4m3);
  const bool act8 = d.act == MLA_ACT_E4M3_DYNAMIC;
  if (act8) {
    if (attend || entry == MLA_ENTRY_KV_UPPROJECT) {
      w.lat8 = take(rows * kL);
      w.lat8_s = take(rows * (kL / 128) * 4);
    }
    if (entry == MLA_ENTRY_PREFILL || entry == MLA_ENTRY_OUT_PROJECT) {
      w.attn8 = take(rows * H * kDv);
      w.attn8_s = take(rows * H * 4);
    }
  } else {
    // bf16 W_o over more than one row tile with a long K: partial tiles of
    // the K-split last wave.
    if (!fp8 && (entry == MLA_ENTRY_PREFILL || entry == MLA_ENTRY_OUT_PROJECT) && rows > 256 &&
        static_cast<int>(H * kDv / 64) >= kSplitMinTileKb)
      w.wo_split = take(static_cast<size_t>(kSplitSlots) * mla::SPLIT_SLOT_FLOATS * 4);
    if (!g_e4m3_onchip) {
      if (fp8 && (attend || copies || entry == MLA_ENTRY_KV_UPPROJECT)) w.wkvb = take(H * (kDn + kDv) * kL * 2);
      if (fp8 && (entry == MLA_ENTRY_PREFILL || copies || entry == MLA_ENTRY_OUT_PROJECT)) w.wo = take(H * kDv * kD * 2);
    } else {
      // On-chip conversion: only the absorbed rows' GEMMs and decode read a
      // bf16 copy of W_kvb (and decode one of W_o).
      const int ng = (static_cast<int>(nq) + 3) / 4;
      if (fp8 && ((attend && w.g_abs < ng) || copies)) w.wkvb = take(H * (kDn + kDv) * kL * 2);
      if (fp8 && copies) w.wo = take(H * kDv * kD * 2);
    }
  }
  w.total = off;
  return w;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

uint8_t* ws_at(void* ws, size_t off) { return static_cast<uint8_t*>(ws) + off; }

// ------------------------------------------------------------------ stage launchers

int launch_dequant(const DeviceState* ds, const void* codes, const float* scale, void* out, int rows, int cols,
                   cudaStream_t st) {
  const int64_t groups = static_cast<int64_t>(rows) * (cols / 16);
  const int64_t want = (groups + 255) / 256;
  const int grid = static_cast<int>(want < int64_t(ds->sms) * 8 ? want : int64_t(ds->sms) * 8);
  return timed_launch(1, st, [&] {
    mla::dequant_e4m3_block128_kernel<<<grid, 256, 0, st>>>(static_cast<const uint8_t*>(codes), scale,
                                                            static_cast<__nv_bfloat16*>(out), rows, cols);
  });
}

constexpr mla::GemmBatch kOneGemm = {1, 0, 0, 0, 0, 0, 0};

template <class Cfg>
int launch_gemm_pair(int pairs_max, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, int M,
                     int N, int K, int* err, int cls, cudaStream_t st, const mla::GemmBatch& bt = kOneGemm,
                     const mla::GemmSplit& sk = mla::kNoSplit) {
  const int tiles = ((M + Cfg::BM - 1) / Cfg::BM) * (N / Cfg::BN) * bt.count;
  const int pairs = tiles < pairs_max ? tiles : pairs_max;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t le = cudaSuccess;
  const int rc = timed_launch(
      cls, st, [&] { le = cudaLaunchKernelEx(&cfg, mla::gemm_bf16_tc2_kernel<Cfg>, ta, tb, tc, M, N, K, bt, sk, err); });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

// v_f16: store the v half of every head as f16 (the attention path's kvh).
int launch_gemm_kvb(const DeviceState* ds, int M, int H, const void* lat, const void* wkvb, void* kvh, bool v_f16,
                    cudaStream_t st) {
  const int N = H * (kDn + kDv), K = kL;
  CUtensorMap ta, tb, tc;
  if (!map_2d(&ta, lat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, K, M, K * 2, 64, 128) ||
      !map_2d(&tb, wkvb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, K, N, K * 2, 64, Gemm2Kvb::HN) ||
      !map_2d(&tc, kvh, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, M, static_cast<uint64_t>(N) * 2, 64, 32))
    return MLA_ERR_CUDA;
  if (v_f16) return launch_gemm_pair<Gemm2KvbAttn>(ds->pairs_kvb, ta, tb, tc, M, N, K, ds->err, 2, st);
  return launch_gemm_pair<Gemm2Kvb>(ds->pairs_kvb, ta, tb, tc, M, N, K, ds->err, 2, st);
}

// K-split of the output projection's last wave (mla::GemmSplit): how many
// last-wave tiles are split (tail) and into how many K ranges (split), for a
// grid of `pairs` CTA pairs. Each range keeps at least kSplitMinKb 64-deep K
// blocks, and tail * split stays within the kSplitSlots partial tiles the
// workspace holds; no split (tail 0) when K is short, the waves are whole or
// fewer than two ranges would result.
mla::GemmSplit wo_split_plan(int tiles, int pairs, int num_kb, float* part) {
  mla::GemmSplit sk = mla::kNoSplit;
  if (part == nullptr || pairs <= 0 || num_kb < kSplitMinTileKb) return sk;
  const int tail = tiles % pairs;
  if (tail == 0) return sk;
  int split = pairs / tail;
  if (split > num_kb / kSplitMinKb) split = num_kb / kSplitMinKb;
  if (split > kSplitSlots / tail) split = kSplitSlots / tail;
  if (split < 2) return sk;
  sk.part = part;
  sk.tail = tail;
  sk.split = split;
  return sk;
}

// split_part: kSplitSlots * SPLIT_SLOT_FLOATS fp32 of workspace for the
// K-split last wave, or nullptr (every tile whole, e.g. so that the result
// matches another kernel's whole-K tiles bit for bit).
int launch_gemm_wo(const DeviceState* ds, int M, int H, const void* attn, const void* wo, void* out,
                   cudaStream_t st, float* split_part = nullptr) {
  const int N = kD, K = H * kDv;
  CUtensorMap ta, tb, tc;
  if (!map_2d(&ta, attn, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, K, M, static_cast<uint64_t>(K) * 2, 64, 128) ||
      !map_2d(&tb, wo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, K, static_cast<uint64_t>(N) * 2, 64, 64) ||
      !map_2d(&tc, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, M, static_cast<uint64_t>(N) * 2, 64, 32))
    return MLA_ERR_CUDA;
  // With a single row tile (decode) the 256-wide tiles would leave most SMs
  // idle while W_o streams through; 128-wide tiles double the pairs.
  if (M <= Gemm2WoNarrow::BM)
    return launch_gemm_pair<Gemm2WoNarrow>(ds->pairs_wo_narrow, ta, tb, tc, M, N, K, ds->err, 4, st);
  const int num_m = (M + Gemm2Wo::BM - 1) / Gemm2Wo::BM, num_n = N / Gemm2Wo::BN;
  const int tiles = num_m * num_n;
  const int pairs = tiles < ds->pairs_wo ? tiles : ds->pairs_wo;
  const mla::GemmSplit sk = wo_split_plan(tiles, pairs, K / Gemm2Wo::BK, split_part);
  int rc = launch_gemm_pair<Gemm2Wo>(ds->pairs_wo, ta, tb, tc, M, N, K, ds->err, 4, st, kOneGemm, sk);
  if (rc != MLA_OK || sk.tail == 0) return rc;
  const int threads = sk.tail * (mla::SPLIT_SLOT_FLOATS / 4);
  return timed_launch(9, st, [&] {
    mla::gemm_split_sum_kernel<<<(threads + 255) / 256, 256, 0, st>>>(
        sk.part, static_cast<__nv_bfloat16*>(out), M, N, num_m, num_n, Gemm2Wo::GROUP_M, tiles - sk.tail, sk.tail,
        sk.split);
  });
}

template <class Cfg>
int launch_gemm_w8t(int pairs_max, const CUtensorMap& tx, const CUtensorMap& tw, const mla::GemmW8tArgs& g, int cls,
                    cudaStream_t st) {
  const int64_t ut = static_cast<int64_t>(Cfg::NT) * Cfg::BN;  // tokens per unit
  const int64_t units = static_cast<int64_t>(g.F / Cfg::BM) * ((g.R + ut - 1) / ut);
  const int pairs = units < pairs_max ? static_cast<int>(units) : pairs_max;
  if (pairs <= 0) return MLA_OK;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t le = cudaSuccess;
  const int rc = timed_launch(cls, st, [&] { le = cudaLaunchKernelEx(&cfg, mla::gemm_bf16_w8t_kernel<Cfg>, tx, tw, g); });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

// kvh = latent . W_kvb^T with W_kvb as e4m3 codes [H*256, 512] and 128 x 128
// block scales, converted on chip (no dequantised copy).
int launch_gemm_w8t_kvb(const DeviceState* ds, int M, int H, const void* lat, const void* wkvb, const float* wkvb_s,
                        void* kvh, bool v_f16, cudaStream_t st) {
  const int N = H * (kDn + kDv), K = kL;
  CUtensorMap tx, tw;
  if (!map_2d(&tx, lat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, K, M, K * 2, 64, GemmW8tKvb::HN) ||
      !map_2d(&tw, wkvb, CU_TENSOR_MAP_DATA_TYPE_UINT8, K, N, K, 64, 128, CU_TENSOR_MAP_SWIZZLE_64B))
    return MLA_ERR_CUDA;
  const mla::GemmW8tArgs g = {wkvb_s, kvh, M, N, K, ds->err};
  if (v_f16) return launch_gemm_w8t<GemmW8tKvbAttn>(ds->pairs_w8t_kvb, tx, tw, g, 2, st);
  return launch_gemm_w8t<GemmW8tKvb>(ds->pairs_w8t_kvb, tx, tw, g, 2, st);
}

// out = attn . W_o with W_o as e4m3 codes [H*128, 7168] and block scales,
// converted on chip.
int launch_gemm_w8t_wo(const DeviceState* ds, int M, int H, const void* attn, const void* wo, const float* wo_s,
                       void* out, cudaStream_t st) {
  const int N = kD, K = H * kDv;
  CUtensorMap tx, tw;
  if (!map_2d(&tx, attn, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, K, M, static_cast<uint64_t>(K) * 2, 64, GemmW8tWo::HN) ||
      !map_2d(&tw, wo, CU_TENSOR_MAP_DATA_TYPE_UINT8, N, K, N, 128, 64, CU_TENSOR_MAP_SWIZZLE_NONE))
    return MLA_ERR_CUDA;
  const mla::GemmW8tArgs g = {wo_s, out, M, N, K, ds->err};
  return launch_gemm_w8t<GemmW8tWo>(ds->pairs_w8t_wo, tx, tw, g, 4, st);
}

// Dynamic e4m3 quantization of a bf16 [rows, cols] matrix: codes [rows, cols],
// scales [cols / 128, rows].
int launch_quant(const void* x, int rows, int cols, void* codes, float* scales, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(rows) * (cols / 128);
  const int64_t per_block = int64_t(2) * mla::kQuantWarps * mla::kQuantItemsPerHalfWarp;
  const unsigned grid = static_cast<unsigned>((items + per_block - 1) / per_block);
  if (grid == 0) return MLA_OK;
  return timed_launch(8, st, [&] {
    mla::quant_e4m3_1x128_kernel<<<grid, 32 * mla::kQuantWarps, 0, st>>>(
        static_cast<const __nv_bfloat16*>(x), rows, cols, static_cast<uint8_t*>(codes), scales);
  });
}

template <class Cfg>
int launch_gemm8_pair(int pairs_max, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, int M,
                      int N, int K, const mla::Gemm8Scales& sc, int* err, int cls, cudaStream_t st) {
  const int tiles = ((M + Cfg::BM - 1) / Cfg::BM) * (N / Cfg::BN);
  const int pairs = tiles < pairs_max ? tiles : pairs_max;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t le = cudaSuccess;
  const int rc = timed_launch(
      cls, st, [&] { le = cudaLaunchKernelEx(&cfg, mla::gemm_e4m3_tc2_kernel<Cfg>, ta, tb, tc, M, N, K, sc, err); });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

// e4m3 up-projection: lat8 codes [M, 512] with scales [4, M] times the e4m3
// W_kvb [H*256, 512] with block scales [2H, 4].
int launch_gemm8_kvb(const DeviceState* ds, int M, int H, const void* lat8, const float* lat_s, const void* wkvb,
                     const float* wkvb_s, void* kvh, bool v_f16, cudaStream_t st) {
  const int N = H * (kDn + kDv), K = kL;
  CUtensorMap ta, tb, tc;
  if (!map_2d(&ta, lat8, CU_TENSOR_MAP_DATA_TYPE_UINT8, K, M, K, 128, 128) ||
      !map_2d(&tb, wkvb, CU_TENSOR_MAP_DATA_TYPE_UINT8, K, N, K, 128, Gemm8Kvb::HN) ||
      !map_2d(&tc, kvh, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, M, static_cast<uint64_t>(N) * 2, 64, 32))
    return MLA_ERR_CUDA;
  const mla::Gemm8Scales sc{lat_s, wkvb_s, 1, K / 128};
  if (v_f16) return launch_gemm8_pair<Gemm8KvbAttn>(ds->pairs8_kvb, ta, tb, tc, M, N, K, sc, ds->err, 2, st);
  return launch_gemm8_pair<Gemm8Kvb>(ds->pairs8_kvb, ta, tb, tc, M, N, K, sc, ds->err, 2, st);
}

// e4m3 output projection: attn8 codes [M, H*128] with scales [H, M] times
// the e4m3 W_o [H*128, 7168] with block scales [H, 56].
int launch_gemm8_wo(const DeviceState* ds, int M, int H, const void* attn8, const float* attn_s, const void* wo,
                    const float* wo_s, void* out, cudaStream_t st) {
  const int N = kD, K = H * kDv;
  CUtensorMap ta, tb, tc;
  if (!map_2d(&ta, attn8, CU_TENSOR_MAP_DATA_TYPE_UINT8, K, M, K, 128, 128) ||
      !map_2d(&tb, wo, CU_TENSOR_MAP_DATA_TYPE_UINT8, N, K, N, Gemm8Wo::HN, 128,
              Gemm8Wo::HN == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map_2d(&tc, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, M, static_cast<uint64_t>(N) * 2, 64, 32))
    return MLA_ERR_CUDA;
  const mla::Gemm8Scales sc{attn_s, wo_s, N / 128, 1};
  return launch_gemm8_pair<Gemm8Wo>(ds->pairs8_wo, ta, tb, tc, M, N, K, sc, ds->err, 4, st);
}

// One launch of the few-row GEMM: 64-row tiles for M <= 64, else 128-row
// tiles (Cfg64 / Cfg128); K columns of A per batch item, or the stream-K
// split of one GEMM over `grid` CTAs.
template <class Cfg64, class Cfg128>
int launch_m64(const DeviceState* ds, const CUtensorMap& ta, const CUtensorMap& tb, int M, int N, int K,
               mla::M64Batch bt, int grid, float* part, void* out, int cls, cudaStream_t st,
               bool dependent = false) {
  const int bm = M <= 64 ? 64 : 128;
  if (g_withhold == kWithholdFewRows) bt.most_tiles = 1;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  cudaError_t le = cudaSuccess;
  const int rc = timed_launch(cls, st, [&] {
    if (bm == 64)
      le = launch_kernel(mla::gemm_m64_kernel<Cfg64>, grid, Cfg64::THREADS, Cfg64::SMEM_BYTES, st, dependent, 1, ta, tb,
                         M, N, K, bt, part, o, ds->err);
    else
      le = launch_kernel(mla::gemm_m64_kernel<Cfg128>, grid, Cfg128::THREADS, Cfg128::SMEM_BYTES, st, dependent, 1, ta,
                         tb, M, N, K, bt, part, o, ds->err);
  });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

// Output projection of M <= 256 rows as a stream-K GEMM (M = 64 or 128 UMMA
// tiles): every CTA takes an equal share of the tiles' k-blocks and writes
// one fp32 partial tile per tile it touches into `part` (room for
// kStreamKCtas + tiles of them); a second kernel sums them into `out`.
int launch_gemm_wo_m64(const DeviceState* ds, int M, int H, const void* attn, const void* wo, float* part,
                       void* out, cudaStream_t st, bool dependent = false) {
  const int N = kD, K = H * kDv;
  const int bm = M <= 64 ? 64 : 128;
  CUtensorMap ta, tb;
  if (!map_2d(&ta, attn, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, K, M, static_cast<uint64_t>(K) * 2, 64, bm) ||
      !map_2d(&tb, wo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, K, static_cast<uint64_t>(N) * 2, 64, 64))
    return MLA_ERR_CUDA;
  const int64_t units = static_cast<int64_t>((M + bm - 1) / bm) * (N / GemmM64::BN) * (K / GemmM64::BK);
  int grid = ds->sms < kStreamKCtas ? ds->sms : kStreamKCtas;
  if (units < grid) grid = static_cast<int>(units);
  const mla::M64Batch bt = {1, 0, 0, 0, 0, 0};
  int rc = launch_m64<GemmM64, GemmM128>(ds, ta, tb, M, N, K, bt, grid, part, nullptr, 4, st, dependent);
  if (rc != MLA_OK) return rc;
  const int blocks = ((M + bm - 1) / bm) * (N / GemmM64::BN) * (bm / mla::kSumRows);
  cudaError_t le = cudaSuccess;
  rc = timed_launch(4, st, [&] {
    le = launch_kernel(mla::sum_segments_kernel, blocks, mla::kSumThreads, 0, st, dependent, 1, part, M, N, K, bm, grid,
                       static_cast<__nv_bfloat16*>(out));
  });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

template <class Cfg64, class Cfg128>
int launch_m64_w8(const DeviceState* ds, const CUtensorMap& ta, const CUtensorMap& tw, int M, int N, int K,
                  mla::M64Batch bt, int grid, const float* scale, float* part, void* out, int cls, cudaStream_t st,
                  bool dependent) {
  if (g_withhold == kWithholdFewRows) bt.most_tiles = 1;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  cudaError_t le = cudaSuccess;
  const int rc = timed_launch(cls, st, [&] {
    if (M <= 64)
      le = launch_kernel(mla::gemm_m64_w8_kernel<Cfg64>, grid, Cfg64::THREADS, Cfg64::SMEM_BYTES, st, dependent, 1, ta, tw,
                         M, N, K, bt, scale, part, o, ds->err);
    else
      le = launch_kernel(mla::gemm_m64_w8_kernel<Cfg128>, grid, Cfg128::THREADS, Cfg128::SMEM_BYTES, st, dependent, 1, ta,
                         tw, M, N, K, bt, scale, part, o, ds->err);
  });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

// launch_gemm_absorb, launch_gemm_unabsorb and launch_gemm_wo_m64 of up to
// kFewRowsE4m3 rows over e4m3 codes. o_lat comes with W_UV's scales multiplied in.
int launch_w8_absorb(const DeviceState* ds, int H, int rows, const void* q_rows, const void* codes, const float* scale,
                     void* qabs, cudaStream_t st) {
  CUtensorMap ta, tw;
  const uint64_t qw = static_cast<uint64_t>(H) * (kDn + kDr);
  if (!map_2d(&ta, q_rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, qw, rows, qw * 2, 64, rows <= 64 ? 64 : 128) ||
      !map_2d(&tw, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, kL, static_cast<uint64_t>(H) * (kDn + kDv), kL, 128, 64,
              CU_TENSOR_MAP_SWIZZLE_NONE))
    return MLA_ERR_CUDA;
  const mla::M64Batch bt = {H, kDn + kDr, 0, kDn + kDv, kL, H * kL};
  const int items = (rows <= 64 ? 1 : (rows + 127) / 128) * (kL / 128) * H;
  return launch_m64_w8<GemmW8Abs64, GemmW8Abs128>(ds, ta, tw, rows, kL, kDn, bt, items < ds->sms ? items : ds->sms, scale,
                                                  nullptr, qabs, 6, st, false);
}

int launch_w8_unabsorb(const DeviceState* ds, int H, int rows, const void* olat, const void* codes, void* attn_rows,
                       cudaStream_t st) {
  CUtensorMap ta, tw;
  if (!map_2d(&ta, olat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(H) * kL, rows,
              static_cast<uint64_t>(H) * kL * 2, 64, rows <= 64 ? 64 : 128) ||
      !map_2d(&tw, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, kL, static_cast<uint64_t>(H) * (kDn + kDv), kL, 64, 128,
              CU_TENSOR_MAP_SWIZZLE_NONE))
    return MLA_ERR_CUDA;
  const mla::M64Batch bt = {H, kL, kDn, kDn + kDv, kDv, H * kDv};
  const int items = (rows <= 64 ? 1 : (rows + 127) / 128) * H;
  return launch_m64_w8<GemmW8Unabs64, GemmW8Unabs128>(ds, ta, tw, rows, kDv, kL, bt, items < ds->sms ? items : ds->sms,
                                                      nullptr, nullptr, attn_rows, 6, st, true);
}

int launch_w8_wo(const DeviceState* ds, int M, int H, const void* attn, const void* codes, const float* scale, float* part,
                 void* out, cudaStream_t st) {
  const int N = kD, K = H * kDv;
  const int bm = M <= 64 ? 64 : 128;
  CUtensorMap ta, tw;
  if (!map_2d(&ta, attn, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, K, M, static_cast<uint64_t>(K) * 2, 64, bm) ||
      !map_2d(&tw, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, N, K, N, 128, 64, CU_TENSOR_MAP_SWIZZLE_NONE))
    return MLA_ERR_CUDA;
  const int64_t units = static_cast<int64_t>((M + bm - 1) / bm) * (N / 128) * (K / 64);
  int grid = ds->sms < kStreamKCtas ? ds->sms : kStreamKCtas;
  if (units < grid) grid = static_cast<int>(units);
  const mla::M64Batch bt = {1, 0, 0, 0, 0, 0};
  int rc = launch_m64_w8<GemmW8Wo64, GemmW8Wo128>(ds, ta, tw, M, N, K, bt, grid, scale, part, nullptr, 4, st, true);
  if (rc != MLA_OK) return rc;
  const int blocks = ((M + bm - 1) / bm) * (N / 128) * (bm / mla::kSumRows);
  cudaError_t le = cudaSuccess;
  rc = timed_launch(4, st, [&] {
    le = launch_kernel(mla::sum_segments_kernel, blocks, mla::kSumThreads, 0, st, true, 1, part, M, N, K, bm, grid,
                       static_cast<__nv_bfloat16*>(out));
  });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

int launch_prepass(const DeviceState* ds, const mla_dims& d, const int32_t* topk, void* bitmap, void* blocks,
                   cudaStream_t st) {
  (void)ds;
  const int nq = (d.T + 127) / 128;
  const int64_t rows = static_cast<int64_t>(d.B) * nq * 128;
  const unsigned grid_rows = static_cast<unsigned>((rows + mla::kPrepassWarps - 1) / mla::kPrepassWarps);
  const size_t smem = static_cast<size_t>(mla::kPrepassWarps) * nq * 4 * 4;
  int rc = timed_launch(0, st, [&] {
    mla::topk_bitmap_rows_kernel<<<grid_rows, 32 * mla::kPrepassWarps, smem, st>>>(
        topk, d.B, d.T, d.topk, nq, static_cast<uint4*>(bitmap));
  });
  if (rc != MLA_OK) return rc;
  dim3 grid((nq + 3) / 4, d.B);
  return timed_launch(0, st, [&] {
    mla::topk_block_list_kernel<<<grid, 32 * mla::kBlockListWarps, 0, st>>>(static_cast<const uint4*>(bitmap), nq,
                                                      static_cast<int32_t*>(blocks));
  });
}

// Block-dense attention for tile groups [0, ngroups_run).
// attn8 / attn8_s set: the output is written as e4m3 codes + scales (the
// input of the e4m3 output projection) instead of bf16.
int launch_attention(const DeviceState* ds, const mla_dims& d, const void* q, const void* kvh, const void* k_pe,
                     const void* bitmap, const void* blocks, float scale, void* attn, int ngroups_run,
                     cudaStream_t st, void* attn8 = nullptr, float* attn8_s = nullptr) {
  // Q tiles and V blocks are 128 rows; each CTA of a pair loads 64 keys of K.
  CUtensorMap tq, tk, tv, tpe;
  const uint64_t kv_inner = static_cast<uint64_t>(d.H) * (kDn + kDv);
  if (!map_3d_bt(&tq, q, static_cast<uint64_t>(d.H) * (kDn + kDr), d.T, d.B) ||
      !map_3d_bt(&tk, kvh, kv_inner, d.T, d.B, 64) || !map_3d_bt(&tv, kvh, kv_inner, d.T, d.B) ||
      !map_3d_bt(&tpe, k_pe, kDr, d.T, d.B, 64))
    return MLA_ERR_CUDA;
  mla::AttnParams p;
  p.B = d.B;
  p.T = d.T;
  p.H = d.H;
  p.nq = (d.T + 127) / 128;
  p.gpitch = (p.nq + 3) / 4;
  p.ngroups = ngroups_run;
  // Heads per scheduling group: the largest of 8, 4, 2, 1 that divides H and
  // keeps the group's K/V (T x 512 bytes per head and batch) near 48 MB or less.
  p.hgroup = 1;
  for (int g = 8; g > 1; g /= 2) {
    if (d.H % g == 0 && static_cast<int64_t>(g) * d.B * d.T * 512 <= (int64_t(48) << 20)) {
      p.hgroup = g;
      break;
    }
  }
  p.scale_log2 = scale * 1.4426950408889634f;
  p.bitmap = static_cast<const uint4*>(bitmap);
  p.blocks = static_cast<const int32_t*>(blocks);
  p.attn = static_cast<__nv_bfloat16*>(attn);
  p.attn8 = static_cast<uint8_t*>(attn8);
  p.attn8_s = attn8_s;
  p.err = ds->err;
  const int64_t pairs = static_cast<int64_t>(d.B) * p.ngroups * d.H;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(mla::kAttnThreads, 1, 1);
  cfg.dynamicSmemBytes = mla::AttnSmem::BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t le = cudaSuccess;
  const int rc = timed_launch(3, st, [&] { le = cudaLaunchKernelEx(&cfg, mla::sparse_mla_attn_kernel, tq, tk, tv, tpe, p); });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

// Selected keys of rows s0 .. s0+rows-1 of batch element b, from the bitmap.
int launch_row_lists(const mla_dims& d, const void* bitmap, int b, int s0, int rows, int kpad, int32_t* lists,
                     int32_t* counts, cudaStream_t st) {
  const int nq = (d.T + 127) / 128;
  const unsigned grid = static_cast<unsigned>((rows + mla::kPrepassWarps - 1) / mla::kPrepassWarps);
  return timed_launch(5, st, [&] {
    mla::topk_row_lists_kernel<<<grid, 32 * mla::kPrepassWarps, 0, st>>>(static_cast<const uint4*>(bitmap), nq, d.T,
                                                                          b, s0, rows, kpad, lists, counts);
  });
}

// Decode: selected cache positions of each sequence's new query.
int launch_decode_lists(const mla_dims& d, const int32_t* topk, int kpad, int32_t* lists, int32_t* counts,
                        cudaStream_t st) {
  return timed_launch(5, st, [&] {
    mla::decode_row_lists_kernel<<<static_cast<unsigned>(d.B), mla::kDecodeListThreads, 0, st>>>(
        topk, d.T, topk ? d.topk : 0, kpad, lists, counts);
  });
}

// q_abs[r, h, :] = q[r, h, 0:128] . W_kvb[h*256 + (0..127), :] for `rows`
// consecutive rows: one GEMM per head (M = rows, N = 512, K = 128).
int launch_gemm_absorb(const DeviceState* ds, int H, int rows, const void* q_rows, const void* wk, void* qabs,
                       cudaStream_t st) {
  CUtensorMap ta, tb, tc;
  const uint64_t qw = static_cast<uint64_t>(H) * (kDn + kDr);
  if (rows <= kFewRows) {
    if (!map_2d(&ta, q_rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, qw, rows, qw * 2, 64, rows <= 64 ? 64 : 128) ||
        !map_2d(&tb, wk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kL, static_cast<uint64_t>(H) * (kDn + kDv), kL * 2, 64, 64))
      return MLA_ERR_CUDA;
    const mla::M64Batch bt = {H, kDn + kDr, 0, kDn + kDv, kL, H * kL};
    const int items = (rows <= 64 ? 1 : (rows + 127) / 128) * (kL / 128) * H;
    return launch_m64<GemmM64Abs, GemmM128Abs>(ds, ta, tb, rows, kL, kDn, bt, items < ds->sms ? items : ds->sms,
                                               nullptr, qabs, 6, st);
  }
  if (!map_2d(&ta, q_rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, qw, rows, qw * 2, 64, 128) ||
      !map_2d(&tb, wk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kL, static_cast<uint64_t>(H) * (kDn + kDv), kL * 2, 64, 64) ||
      !map_2d(&tc, qabs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(H) * kL, rows,
              static_cast<uint64_t>(H) * kL * 2, 64, 32))
    return MLA_ERR_CUDA;
  const mla::GemmBatch bt = {H, 0, kDn + kDr, 0, kDn + kDv, 0, kL};
  return launch_gemm_pair<Gemm2Wo>(ds->pairs_wo, ta, tb, tc, rows, kL, kDn, ds->err, 6, st, bt);
}

// attn[r, h, :] = o_lat[r, h, :] . W_kvb[h*256 + 128 + (0..127), :]^T: one
// GEMM per head (M = rows, N = 128, K = 512).
int launch_gemm_unabsorb(const DeviceState* ds, int H, int rows, const void* olat, const void* wk, void* attn_rows,
                         cudaStream_t st, bool dependent = false) {
  CUtensorMap ta, tb, tc;
  if (rows <= kFewRows) {
    if (!map_2d(&ta, olat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(H) * kL, rows,
                static_cast<uint64_t>(H) * kL * 2, 64, rows <= 64 ? 64 : 128) ||
        !map_2d(&tb, wk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kL, static_cast<uint64_t>(H) * (kDn + kDv), kL * 2, 64,
                128))
      return MLA_ERR_CUDA;
    const mla::M64Batch bt = {H, kL, kDn, kDn + kDv, kDv, H * kDv};
    const int items = (rows <= 64 ? 1 : (rows + 127) / 128) * H;
    return launch_m64<GemmM64Unabs, GemmM128Unabs>(ds, ta, tb, rows, kDv, kL, bt, items < ds->sms ? items : ds->sms,
                                                   nullptr, attn_rows, 6, st, dependent);
  }
  if (!map_2d(&ta, olat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(H) * kL, rows,
              static_cast<uint64_t>(H) * kL * 2, 64, 128) ||
      !map_2d(&tb, wk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kL, static_cast<uint64_t>(H) * (kDn + kDv), kL * 2, 64,
              Gemm2Unabs::HN) ||
      !map_2d(&tc, attn_rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(H) * kDv, rows,
              static_cast<uint64_t>(H) * kDv * 2, 64, 32))
    return MLA_ERR_CUDA;
  const mla::GemmBatch bt = {H, 0, kL, kDn, kDn + kDv, 0, kDv};
  return launch_gemm_pair<Gemm2Unabs>(ds->pairs_unabs, ta, tb, tc, rows, kDv, kL, ds->err, 6, st, bt);
}

// Absorbed attention for `rows` rows (one CTA per row and group of 64 heads).
int launch_attention_absorbed(const DeviceState* ds, const mla_dims& d, const void* lat, const void* k_pe, int rows,
                              int key_row0, int rows_per_seq, int seq_stride, int kpad, const int32_t* lists,
                              const int32_t* counts, const void* qabs,
                              const void* q_rows, void* olat, float scale, cudaStream_t st, int parts = 1,
                              void* part_ml = nullptr, void* part_o = nullptr) {
  mla::AbsParams p;
  p.rows = rows;
  p.H = d.H;
  p.kpad = kpad;
  p.key_row0 = key_row0;
  p.rows_per_seq = rows_per_seq;
  p.seq_stride = seq_stride;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.lists = lists;
  p.counts = counts;
  p.qabs = static_cast<const __nv_bfloat16*>(qabs);
  p.q = static_cast<const __nv_bfloat16*>(q_rows);
  p.lat = static_cast<const __nv_bfloat16*>(lat);
  p.kpe = static_cast<const __nv_bfloat16*>(k_pe);
  p.olat = static_cast<__nv_bfloat16*>(olat);
  p.parts = parts;
  p.part_ml = static_cast<float2*>(part_ml);
  p.part_o = static_cast<__nv_bfloat16*>(part_o);
  p.err = ds->err;
  int rc = timed_launch(7, st, [&] {
    mla::absorbed_attn_kernel<<<static_cast<unsigned>(rows * ((d.H + 63) / 64) * parts), mla::kAbsThreads,
                                 mla::AbsSmem::BYTES, st>>>(p);
  });
  if (rc != MLA_OK || parts == 1) return rc;
  const int64_t items = static_cast<int64_t>(rows) * d.H;
  return timed_launch(7, st, [&] {
    mla::absorbed_combine_kernel<<<static_cast<unsigned>((items + mla::kCombineWarps - 1) / mla::kCombineWarps),
                                    32 * mla::kCombineWarps, 0, st>>>(p);
  });
}

}  // namespace

// ------------------------------------------------------------------ C ABI

namespace {

int begin_call(const mla_dims* dims, int entry, bool has_topk, void* ws, size_t ws_bytes, DeviceState** ds,
               WsLayout* lay) {
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  *lay = ws_layout(*dims, entry, has_topk);
  if (lay->total > 0 && (ws == nullptr || ws_bytes < lay->total)) return MLA_ERR_WORKSPACE;
  if (ws != nullptr && !aligned16(ws)) return MLA_ERR_ALIGN;
  return device_state(ds);
}

// Up-projection into kvh; dequantises W_kvb into the workspace first when
// it is stored as e4m3.
int run_upproject(const DeviceState* ds, const mla_dims& d, const WsLayout& lay, void* ws, const void* lat,
                  const void* W_kvb, const float* W_kvb_scale, void* kvh, bool v_f16, cudaStream_t st) {
  if (d.act == MLA_ACT_E4M3_DYNAMIC) {
    const int M = d.B * d.T;
    void* lat8 = ws_at(ws, lay.lat8);
    float* lat_s = reinterpret_cast<float*>(ws_at(ws, lay.lat8_s));
    int rc = launch_quant(lat, M, kL, lat8, lat_s, st);
    if (rc != MLA_OK) return rc;
    return launch_gemm8_kvb(ds, M, d.H, lat8, lat_s, W_kvb, W_kvb_scale, kvh, v_f16, st);
  }
  const void* wk = W_kvb;
  if (d.wdtype == MLA_W_E4M3_BLOCK128) {
    if (g_e4m3_onchip) return launch_gemm_w8t_kvb(ds, d.B * d.T, d.H, lat, W_kvb, W_kvb_scale, kvh, v_f16, st);
    void* dq = ws_at(ws, lay.wkvb);
    int rc = launch_dequant(ds, W_kvb, W_kvb_scale, dq, d.H * (kDn + kDv), kL, st);
    if (rc != MLA_OK) return rc;
    wk = dq;
  }
  return launch_gemm_kvb(ds, d.B * d.T, d.H, lat, wk, kvh, v_f16, st);
}

int run_attend(const DeviceState* ds, const mla_dims& d, const WsLayout& lay, void* ws, const void* q,
               const void* lat, const void* k_pe, const void* W_kvb, const float* W_kvb_scale,
               const int32_t* topk_idx, float scale, void* attn, cudaStream_t st, void* attn8 = nullptr,
               float* attn8_s = nullptr) {
  const int nq = (d.T + 127) / 128;
  const int ng = (nq + 3) / 4;
  const void* wk = W_kvb;
  int rc = MLA_OK;
  const bool act8 = d.act == MLA_ACT_E4M3_DYNAMIC;  // every row block-dense (absorbed_first_group)
  // e4m3 W_kvb with bf16 activations: dequantised once into the workspace for
  // every GEMM of the call, or, with on-chip conversion, only for the
  // absorbed rows' absorb / un-absorb GEMMs (which read it as bf16).
  const bool onchip = d.wdtype == MLA_W_E4M3_BLOCK128 && !act8 && g_e4m3_onchip;
  if (d.wdtype == MLA_W_E4M3_BLOCK128 && !act8 && (!onchip || lay.g_abs < ng)) {
    void* dq = ws_at(ws, lay.wkvb);
    rc = launch_dequant(ds, W_kvb, W_kvb_scale, dq, d.H * (kDn + kDv), kL, st);
    if (rc != MLA_OK) return rc;
    wk = dq;
  }
  void* kvh = nullptr;
  if (lay.g_abs > 0) {  // up-projected keys, for the block-dense rows only
    kvh = ws_at(ws, lay.kvh);
    rc = (act8 || onchip) ? run_upproject(ds, d, lay, ws, lat, W_kvb, W_kvb_scale, kvh, /*v_f16=*/true, st)
                          : launch_gemm_kvb(ds, d.B * d.T, d.H, lat, wk, kvh, /*v_f16=*/true, st);
    if (rc != MLA_OK) return rc;
  }
  void* bitmap = nullptr;
  void* blocks = nullptr;
  if (topk_idx != nullptr) {
    bitmap = ws_at(ws, lay.bitmap);
    blocks = ws_at(ws, lay.blocks);
    rc = launch_prepass(ds, d, topk_idx, bitmap, blocks, st);
    if (rc != MLA_OK) return rc;
  }
  if (lay.g_abs > 0) {
    rc = launch_attention(ds, d, q, kvh, k_pe, bitmap, blocks, scale, attn, lay.g_abs, st, attn8, attn8_s);
    if (rc != MLA_OK) return rc;
  }
  if (lay.g_abs >= ng) return MLA_OK;
  // Absorbed rows [512 * g_abs, T) of every batch element, in passes.
  void* qabs = ws_at(ws, lay.qabs);
  void* olat = ws_at(ws, lay.olat);
  int32_t* lists = reinterpret_cast<int32_t*>(ws_at(ws, lay.lists));
  int32_t* counts = reinterpret_cast<int32_t*>(ws_at(ws, lay.counts));
  const size_t qrow = static_cast<size_t>(d.H) * (kDn + kDr) * 2, arow = static_cast<size_t>(d.H) * kDv * 2;
  for (int b = 0; b < d.B; ++b) {
    for (int s0 = 512 * lay.g_abs; s0 < d.T; s0 += lay.abs_chunk) {
      const int rows = d.T - s0 < lay.abs_chunk ? d.T - s0 : lay.abs_chunk;
      const size_t r0 = static_cast<size_t>(b) * d.T + s0;
      const void* q_rows = static_cast<const uint8_t*>(q) + r0 * qrow;
      void* attn_rows = static_cast<uint8_t*>(attn) + r0 * arow;
      if ((rc = launch_row_lists(d, bitmap, b, s0, rows, lay.kpad, lists, counts, st)) != MLA_OK) return rc;
      if ((rc = launch_gemm_absorb(ds, d.H, rows, q_rows, wk, qabs, st)) != MLA_OK) return rc;
      if ((rc = launch_attention_absorbed(ds, d, lat, k_pe, rows, b * d.T, rows, 0, lay.kpad, lists, counts, qabs,
                                          q_rows, olat, scale, st)) != MLA_OK)
        return rc;
      if ((rc = launch_gemm_unabsorb(ds, d.H, rows, olat, wk, attn_rows, st)) != MLA_OK) return rc;
    }
  }
  return MLA_OK;
}

int run_out_project(const DeviceState* ds, const mla_dims& d, const WsLayout& lay, void* ws, const void* attn,
                    const void* W_o, const float* W_o_scale, void* out, cudaStream_t st) {
  if (d.act == MLA_ACT_E4M3_DYNAMIC) {
    const int M = d.B * d.T;
    void* attn8 = ws_at(ws, lay.attn8);
    float* attn_s = reinterpret_cast<float*>(ws_at(ws, lay.attn8_s));
    int rc = launch_quant(attn, M, d.H * kDv, attn8, attn_s, st);
    if (rc != MLA_OK) return rc;
    return launch_gemm8_wo(ds, M, d.H, attn8, attn_s, W_o, W_o_scale, out, st);
  }
  const void* wo = W_o;
  if (d.wdtype == MLA_W_E4M3_BLOCK128 && g_e4m3_onchip)
    return launch_gemm_w8t_wo(ds, d.B * d.T, d.H, attn, W_o, W_o_scale, out, st);
  if (d.wdtype == MLA_W_E4M3_BLOCK128) {
    // Whole-K tiles only, so that both e4m3 conversion modes give the same bits.
    void* dq = ws_at(ws, lay.wo);
    int rc = launch_dequant(ds, W_o, W_o_scale, dq, d.H * kDv, kD, st);
    if (rc != MLA_OK) return rc;
    return launch_gemm_wo(ds, d.B * d.T, d.H, attn, dq, out, st);
  }
  float* split = lay.wo_split == kNone ? nullptr : reinterpret_cast<float*>(ws_at(ws, lay.wo_split));
  return launch_gemm_wo(ds, d.B * d.T, d.H, attn, wo, out, st, split);
}

// Decode: one new query per sequence (row s = T-1) against the cache, in the
// absorbed form.
int run_decode(const DeviceState* ds, const mla_dims& d, const WsLayout& lay, void* ws, const void* q,
               const void* lat, const void* k_pe, const void* W_kvb, const float* W_kvb_scale, const void* W_o,
               const float* W_o_scale, const int32_t* topk_idx, float scale, void* out, cudaStream_t st) {
  const void* wk = W_kvb;
  int rc = MLA_OK;
  if (d.wdtype == MLA_W_E4M3_BLOCK128) {
    void* dq = ws_at(ws, lay.wkvb);
    if ((rc = launch_dequant(ds, W_kvb, W_kvb_scale, dq, d.H * (kDn + kDv), kL, st)) != MLA_OK) return rc;
    wk = dq;
  }
  void* qabs = ws_at(ws, lay.qabs);
  void* olat = ws_at(ws, lay.olat);
  void* attn = ws_at(ws, lay.attn);
  int32_t* lists = reinterpret_cast<int32_t*>(ws_at(ws, lay.lists));
  int32_t* counts = reinterpret_cast<int32_t*>(ws_at(ws, lay.counts));
  if ((rc = launch_decode_lists(d, topk_idx, lay.kpad, lists, counts, st)) != MLA_OK) return rc;
  if ((rc = launch_gemm_absorb(ds, d.H, d.B, q, wk, qabs, st)) != MLA_OK) return rc;
  if ((rc = launch_attention_absorbed(ds, d, lat, k_pe, d.B, 0, 1, d.T, lay.kpad, lists, counts, qabs, q, olat, scale,
                                      st, lay.parts, lay.parts > 1 ? ws_at(ws, lay.part_ml) : nullptr,
                                      lay.parts > 1 ? ws_at(ws, lay.part_o) : nullptr)) != MLA_OK)
    return rc;
  if ((rc = launch_gemm_unabsorb(ds, d.H, d.B, olat, wk, attn, st)) != MLA_OK) return rc;
  const void* wo = W_o;
  if (d.wdtype == MLA_W_E4M3_BLOCK128) {
    void* dq = ws_at(ws, lay.wo);
    if ((rc = launch_dequant(ds, W_o, W_o_scale, dq, d.H * kDv, kD, st)) != MLA_OK) return rc;
    wo = dq;
  }
  if (lay.wo_part != kNone)
    return launch_gemm_wo_m64(ds, d.B, d.H, attn, wo, reinterpret_cast<float*>(ws_at(ws, lay.wo_part)), out, st);
  return launch_gemm_wo(ds, d.B, d.H, attn, wo, out, st);
}

// ------------------------------------------------------------------ paged serving

constexpr int64_t kMaxCacheRows = int64_t(1) << 30;  // rows of one layer's cache, positions of one table row
constexpr int64_t kMaxQueryRows = int64_t(1) << 27;   // (node, head) rows of one call: 32-bit coordinates and grids
constexpr int kMaxLayers = 65535;                    // a grid dimension

int check_pages(const mla_pages* pg, bool table) {
  if (pg == nullptr) return MLA_ERR_NULL;
  if (pg->num_pages < 0 || pg->page_size < 16 || (pg->page_size & (pg->page_size - 1)) != 0) return MLA_ERR_SHAPE;
  if (static_cast<int64_t>(pg->num_pages) * pg->page_size > kMaxCacheRows) return MLA_ERR_SHAPE;
  if (pg->layers < 1 || pg->layers > kMaxLayers) return MLA_ERR_SHAPE;
  if (table && (pg->table_width < 1 || static_cast<int64_t>(pg->table_width) * pg->page_size > kMaxCacheRows))
    return MLA_ERR_SHAPE;
  return MLA_OK;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

mla::RopeTable rope_table(const mla_rope_table& t) {
  mla::RopeTable r;
  for (int i = 0; i < mla::kRopePairs; ++i) r.turns[i] = t.turns[i];
  r.magnitude = t.magnitude;
  r.layout = t.layout;
  return r;
}

// Attention of B trees of N nodes over the pages: q_abs (in the workspace) and
// q's rotary part against the cache, into o_lat (in the workspace), times
// W_UV's block scales if v_scale (W_kvb's scales) is given.
int launch_tree_attention(const DeviceState* ds, const mla_dims& d, const mla_pages& pg, const WsLayout& lay, void* ws,
                          const void* q, const void* kv, const void* pe, const int32_t* table,
                          const int32_t* cache_len, const int32_t* n_nodes, const int32_t* parents, float scale,
                          const float* v_scale, cudaStream_t st, bool dependent) {
  mla::TreeParams p = {};
  p.B = d.B;
  p.N = d.T;
  p.H = d.H;
  p.num_pages = pg.num_pages;
  p.page_shift = log2_of(pg.page_size);
  p.table_width = pg.table_width;
  p.box_shift = p.page_shift < 6 ? p.page_shift : 6;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.kv = static_cast<const uint4*>(kv);
  p.table = table;
  p.cache_len = cache_len;
  p.n_nodes = n_nodes;
  p.parents = parents;
  p.v_scale = v_scale;
  p.olat = reinterpret_cast<__nv_bfloat16*>(ws_at(ws, lay.olat));
  p.ustart = reinterpret_cast<int64_t*>(ws_at(ws, lay.tree_start));
  p.part_o = reinterpret_cast<float*>(ws_at(ws, lay.tree_o));
  p.part_ml = reinterpret_cast<float2*>(ws_at(ws, lay.tree_ml));
  p.most_blocks = g_withhold == kWithholdTree ? 1 : 0x7fffffff;
  p.err = ds->err;
  const uint64_t qrows = static_cast<uint64_t>(d.B) * d.T * d.H, crows = static_cast<uint64_t>(pg.num_pages) * pg.page_size;
  const uint32_t box = 1u << p.box_shift;
  CUtensorMap tkv, tpe, tqa, tq;
  if (!map_chunks(&tkv, kv, crows, box, box == 64 ? 2 : 1) ||
      !map_2d(&tpe, pe, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDr, crows, kDr * 2, 64, box) ||
      !map_chunks(&tqa, ws_at(ws, lay.qabs), qrows, 64, 2) ||
      !map_2d(&tq, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDn + kDr, qrows, (kDn + kDr) * 2, 64, 64))
    return MLA_ERR_CUDA;
  cudaError_t le = cudaSuccess;
  int rc = timed_launch(7, st, [&] {
    le = launch_kernel(mla::tree_attn_kernel, 2 * ds->pairs_tree, mla::kTreeThreads, mla::TreeSmem::BYTES, st, dependent, 2,
                       tkv, tpe, tqa, tq, p);
  });
  if (le != cudaSuccess) return MLA_ERR_CUDA;
  if (rc != MLA_OK) return rc;
  const int64_t tiles = static_cast<int64_t>(d.B) * ((d.T * d.H + mla::kTreeRows - 1) / mla::kTreeRows);
  using Many = mla::TreeJoin<16, 1>;
  using Some = mla::TreeJoin<4, 1>;
  using Few = mla::TreeJoin<4, 4>;
  rc = timed_launch(7, st, [&] {
    auto join = [&](auto kernel, int64_t blocks, int threads) {
      le = launch_kernel(kernel, static_cast<unsigned>(tiles * blocks), threads, 0, st, dependent, 1, p, ds->pairs_tree);
    };
    if (tiles * Few::BLOCKS <= 2 * ds->sms)
      join(mla::tree_combine_kernel<4, 4>, Few::BLOCKS, Few::THREADS);
    else if (tiles * Many::BLOCKS < 2 * ds->sms)
      join(mla::tree_combine_kernel<4, 1>, Some::BLOCKS, Some::THREADS);
    else
      join(mla::tree_combine_kernel<16, 1>, Many::BLOCKS, Many::THREADS);
  });
  return le != cudaSuccess ? MLA_ERR_CUDA : rc;
}

// One decoding step of B trees of N nodes.
int run_tree_decode(const DeviceState* ds, const mla_dims& d, const mla_pages& pg, const WsLayout& lay, void* ws,
                    const void* q, const void* kv, const void* pe, const int32_t* table, const int32_t* cache_len,
                    const int32_t* n_nodes, const int32_t* parents, const void* W_kvb, const float* W_kvb_scale,
                    const void* W_o, const float* W_o_scale, float scale, void* out, cudaStream_t st) {
  const int rows = d.B * d.T;
  const bool e4m3 = d.wdtype == MLA_W_E4M3_BLOCK128, few = rows <= tree_few_rows(e4m3);
  void* qabs = ws_at(ws, lay.qabs);
  void* olat = ws_at(ws, lay.olat);
  void* attn = ws_at(ws, lay.attn);
  int rc = MLA_OK;
  if (few) {
    // After the first, each kernel is launched as a dependent of the one before,
    // so that its set-up runs while that one ends.
    float* part = reinterpret_cast<float*>(ws_at(ws, lay.wo_part));
    rc = e4m3 ? launch_w8_absorb(ds, d.H, rows, q, W_kvb, W_kvb_scale, qabs, st)
              : launch_gemm_absorb(ds, d.H, rows, q, W_kvb, qabs, st);
    if (rc != MLA_OK) return rc;
    if ((rc = launch_tree_attention(ds, d, pg, lay, ws, q, kv, pe, table, cache_len, n_nodes, parents, scale,
                                    e4m3 ? W_kvb_scale : nullptr, st, true)) != MLA_OK)
      return rc;
    rc = e4m3 ? launch_w8_unabsorb(ds, d.H, rows, olat, W_kvb, attn, st)
              : launch_gemm_unabsorb(ds, d.H, rows, olat, W_kvb, attn, st, true);
    if (rc != MLA_OK) return rc;
    return e4m3 ? launch_w8_wo(ds, rows, d.H, attn, W_o, W_o_scale, part, out, st)
                : launch_gemm_wo_m64(ds, rows, d.H, attn, W_o, part, out, st, true);
  }
  // More rows: the pair GEMMs, over bf16 copies of e4m3 weights.
  const void* wk = W_kvb;
  const void* wo = W_o;
  if (e4m3) {
    void* dk = ws_at(ws, lay.wkvb);
    void* dw = ws_at(ws, lay.wo);
    if ((rc = launch_dequant(ds, W_kvb, W_kvb_scale, dk, d.H * (kDn + kDv), kL, st)) != MLA_OK) return rc;
    if ((rc = launch_dequant(ds, W_o, W_o_scale, dw, d.H * kDv, kD, st)) != MLA_OK) return rc;
    wk = dk;
    wo = dw;
  }
  if ((rc = launch_gemm_absorb(ds, d.H, rows, q, wk, qabs, st)) != MLA_OK) return rc;
  if ((rc = launch_tree_attention(ds, d, pg, lay, ws, q, kv, pe, table, cache_len, n_nodes, parents, scale, nullptr, st,
                                  false)) != MLA_OK)
    return rc;
  if ((rc = launch_gemm_unabsorb(ds, d.H, rows, olat, wk, attn, st)) != MLA_OK) return rc;
  return launch_gemm_wo(ds, rows, d.H, attn, wo, out, st);
}

bool fp8_scales_ok(const mla_dims* d, const float* s) { return d->wdtype != MLA_W_E4M3_BLOCK128 || s != nullptr; }

}  // namespace

extern "C" {

size_t mla_workspace_bytes(const mla_dims* dims, int entry, int has_topk) {
  if (check_dims(dims) != MLA_OK || entry < MLA_ENTRY_KV_UPPROJECT || entry > MLA_ENTRY_TREE_DECODE) return 0;
  if ((entry == MLA_ENTRY_DECODE || entry == MLA_ENTRY_TREE_DECODE) && dims->act != MLA_ACT_BF16) return 0;
  if (entry == MLA_ENTRY_TREE_DECODE &&
      (dims->topk != 0 || dims->T > MLA_MAX_TREE || static_cast<int64_t>(dims->B) * dims->T * dims->H > kMaxQueryRows))
    return 0;
  return ws_layout(*dims, entry, has_topk != 0).total;
}

int mla_kv_upproject(const mla_dims* dims, const void* kv_latent, const void* W_kvb, const float* W_kvb_scale,
                     void* kvh_out, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  DeviceState* ds = nullptr;
  WsLayout lay;
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  if (!kv_latent || !W_kvb || !kvh_out || !fp8_scales_ok(dims, W_kvb_scale)) return MLA_ERR_NULL;
  if (!aligned16(kv_latent) || !aligned16(W_kvb) || !aligned16(kvh_out) || !aligned16(W_kvb_scale))
    return MLA_ERR_ALIGN;
  rc = begin_call(dims, MLA_ENTRY_KV_UPPROJECT, false, workspace, ws_bytes, &ds, &lay);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  return run_upproject(ds, *dims, lay, workspace, kv_latent, W_kvb, W_kvb_scale, kvh_out, /*v_f16=*/false,
                       reinterpret_cast<cudaStream_t>(stream));
}

int mla_attend(const mla_dims* dims, const void* q, const void* kv_latent, const void* k_pe, const void* W_kvb,
               const float* W_kvb_scale, const int32_t* topk_idx, float scale, void* attn_out, void* workspace,
               size_t ws_bytes, mla_stream_t stream) {
  DeviceState* ds = nullptr;
  WsLayout lay;
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  if (!q || !kv_latent || !k_pe || !W_kvb || !attn_out || !fp8_scales_ok(dims, W_kvb_scale)) return MLA_ERR_NULL;
  if (topk_idx != nullptr && dims->topk < 1) return MLA_ERR_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv_latent) || !aligned16(k_pe) || !aligned16(W_kvb) || !aligned16(attn_out) ||
      !aligned16(W_kvb_scale) || !aligned16(topk_idx))
    return MLA_ERR_ALIGN;
  rc = begin_call(dims, MLA_ENTRY_ATTEND, topk_idx != nullptr, workspace, ws_bytes, &ds, &lay);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  return run_attend(ds, *dims, lay, workspace, q, kv_latent, k_pe, W_kvb, W_kvb_scale, topk_idx, scale, attn_out,
                    reinterpret_cast<cudaStream_t>(stream));
}

int mla_out_project(const mla_dims* dims, const void* attn, const void* W_o, const float* W_o_scale, void* out,
                    void* workspace, size_t ws_bytes, mla_stream_t stream) {
  DeviceState* ds = nullptr;
  WsLayout lay;
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  if (!attn || !W_o || !out || !fp8_scales_ok(dims, W_o_scale)) return MLA_ERR_NULL;
  if (!aligned16(attn) || !aligned16(W_o) || !aligned16(out) || !aligned16(W_o_scale)) return MLA_ERR_ALIGN;
  rc = begin_call(dims, MLA_ENTRY_OUT_PROJECT, false, workspace, ws_bytes, &ds, &lay);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  return run_out_project(ds, *dims, lay, workspace, attn, W_o, W_o_scale, out,
                         reinterpret_cast<cudaStream_t>(stream));
}

int mla_prefill(const mla_dims* dims, const void* q, const void* kv_latent, const void* k_pe, const void* W_kvb,
                const float* W_kvb_scale, const void* W_o, const float* W_o_scale, const int32_t* topk_idx,
                float scale, void* out, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  DeviceState* ds = nullptr;
  WsLayout lay;
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  if (!q || !kv_latent || !k_pe || !W_kvb || !W_o || !out || !fp8_scales_ok(dims, W_kvb_scale) ||
      !fp8_scales_ok(dims, W_o_scale))
    return MLA_ERR_NULL;
  if (topk_idx != nullptr && dims->topk < 1) return MLA_ERR_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv_latent) || !aligned16(k_pe) || !aligned16(W_kvb) || !aligned16(W_o) ||
      !aligned16(out) || !aligned16(W_kvb_scale) || !aligned16(W_o_scale) || !aligned16(topk_idx))
    return MLA_ERR_ALIGN;
  rc = begin_call(dims, MLA_ENTRY_PREFILL, topk_idx != nullptr, workspace, ws_bytes, &ds, &lay);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dims->act == MLA_ACT_E4M3_DYNAMIC) {
    // The attention kernel writes its output already quantized (every row
    // is block-dense with e4m3 activations), so W_o reads the codes directly.
    void* attn8 = ws_at(workspace, lay.attn8);
    float* attn8_s = reinterpret_cast<float*>(ws_at(workspace, lay.attn8_s));
    rc = run_attend(ds, *dims, lay, workspace, q, kv_latent, k_pe, W_kvb, W_kvb_scale, topk_idx, scale, nullptr, st,
                    attn8, attn8_s);
    if (rc != MLA_OK) return rc;
    return launch_gemm8_wo(ds, dims->B * dims->T, dims->H, attn8, attn8_s, W_o, W_o_scale, out, st);
  }
  void* attn = ws_at(workspace, lay.attn);
  rc = run_attend(ds, *dims, lay, workspace, q, kv_latent, k_pe, W_kvb, W_kvb_scale, topk_idx, scale, attn, st);
  if (rc != MLA_OK) return rc;
  return run_out_project(ds, *dims, lay, workspace, attn, W_o, W_o_scale, out, st);
}

int mla_decode(const mla_dims* dims, const void* q, const void* kv_latent, const void* k_pe, const void* W_kvb,
               const float* W_kvb_scale, const void* W_o, const float* W_o_scale, const int32_t* topk_idx,
               float scale, void* out, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  DeviceState* ds = nullptr;
  WsLayout lay;
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  if (!q || !kv_latent || !k_pe || !W_kvb || !W_o || !out || !fp8_scales_ok(dims, W_kvb_scale) ||
      !fp8_scales_ok(dims, W_o_scale))
    return MLA_ERR_NULL;
  if (topk_idx != nullptr && dims->topk < 1) return MLA_ERR_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv_latent) || !aligned16(k_pe) || !aligned16(W_kvb) || !aligned16(W_o) ||
      !aligned16(out) || !aligned16(W_kvb_scale) || !aligned16(W_o_scale) || !aligned16(topk_idx))
    return MLA_ERR_ALIGN;
  if (dims->act != MLA_ACT_BF16) return MLA_ERR_UNSUPPORTED;
  rc = begin_call(dims, MLA_ENTRY_DECODE, topk_idx != nullptr, workspace, ws_bytes, &ds, &lay);
  if (rc != MLA_OK) return rc;
  return run_decode(ds, *dims, lay, workspace, q, kv_latent, k_pe, W_kvb, W_kvb_scale, W_o, W_o_scale, topk_idx,
                    scale, out, reinterpret_cast<cudaStream_t>(stream));
}

int mla_quantize_act(const void* x, int rows, int cols, void* codes, float* scales, mla_stream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 128 != 0) return MLA_ERR_SHAPE;
  if (static_cast<int64_t>(rows) * cols >= (int64_t(1) << 40)) return MLA_ERR_SHAPE;
  if (rows == 0) return MLA_OK;
  if (!x || !codes || !scales) return MLA_ERR_NULL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MLA_ERR_ALIGN;
  DeviceState* ds = nullptr;
  const int rc = device_state(&ds);
  if (rc != MLA_OK) return rc;
  return launch_quant(x, rows, cols, codes, scales, reinterpret_cast<cudaStream_t>(stream));
}

int mla_rope_init(mla_rope_table* table, int layout, double base, int scaling, double factor, double original_len,
                  double beta_fast, double beta_slow, float magnitude) {
  if (table == nullptr) return MLA_ERR_NULL;
  if (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF) return MLA_ERR_UNSUPPORTED;
  if (scaling != MLA_ROPE_UNSCALED && scaling != MLA_ROPE_LINEAR && scaling != MLA_ROPE_YARN)
    return MLA_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !std::isfinite(base) || !std::isfinite(magnitude)) return MLA_ERR_SHAPE;
  if (scaling != MLA_ROPE_UNSCALED && (!(factor >= 1.0) || !std::isfinite(factor))) return MLA_ERR_SHAPE;
  // 64-bit mantissas throughout: a double's would be 2^-54 of a frequency off, 2^8
  // units of the table.
  const long double two_pi = 2.0L * 3.14159265358979323846264338328L, b = base, dim = mla::kRopeDim;
  long double lo = 0.0L, hi = 0.0L;
  if (scaling == MLA_ROPE_YARN) {
    if (!(original_len > 0.0) || !std::isfinite(original_len) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
        !std::isfinite(beta_fast))
      return MLA_ERR_SHAPE;
    auto at = [&](double turns) { return dim * std::log(original_len / (two_pi * turns)) / (2.0L * std::log(b)); };
    lo = std::fmax(std::floor(at(beta_fast)), 0.0L);
    hi = std::fmin(std::ceil(at(beta_slow)), dim - 1.0L);
  }
  for (int i = 0; i < mla::kRopePairs; ++i) {
    long double f = std::pow(b, -2.0L * i / dim);
    if (scaling == MLA_ROPE_LINEAR) f /= factor;
    if (scaling == MLA_ROPE_YARN) {
      const long double r = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3L), 0.0L), 1.0L);
      f = f * (1.0L - r) + f / factor * r;
    }
    // f <= 1 radian per position, so the fraction of a turn fits (2^64 / 2 pi < 2^62)
    table->turns[i] = static_cast<uint64_t>(f / two_pi * 18446744073709551616.0L + 0.5L);
  }
  table->magnitude = magnitude;
  table->layout = layout;
  return MLA_OK;
}

int mla_rope(const mla_rope_table* table, const void* x, long long x_row_stride, long long x_head_stride, void* out,
             long long out_row_stride, long long out_head_stride, int rows, int heads, int width, int offset,
             const int32_t* positions, int inverse, mla_stream_t stream) {
  if (table == nullptr) return MLA_ERR_NULL;
  if (table->layout != MLA_ROPE_INTERLEAVED && table->layout != MLA_ROPE_HALF) return MLA_ERR_UNSUPPORTED;
  if (rows < 0 || heads < 0 || width < mla::kRopeDim || width > 2048 || width % 8 != 0) return MLA_ERR_SHAPE;
  if (offset < 0 || offset % 8 != 0 || offset + mla::kRopeDim > width) return MLA_ERR_SHAPE;
  if ((inverse != 0 && inverse != 1) || x_row_stride % 8 != 0 || x_head_stride % 8 != 0 || out_row_stride % 8 != 0 ||
      out_head_stride % 8 != 0)
    return MLA_ERR_SHAPE;
  if (rows == 0 || heads == 0) return MLA_OK;
  if (!x || !out || !positions) return MLA_ERR_NULL;
  if (!aligned16(x) || !aligned16(out) || (reinterpret_cast<uintptr_t>(positions) & 3u)) return MLA_ERR_ALIGN;
  DeviceState* ds = nullptr;
  const int rc = device_state(&ds);
  if (rc != MLA_OK) return rc;
  mla::RopeParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.x_row = x_row_stride;
  p.x_head = x_head_stride;
  p.o_row = out_row_stride;
  p.o_head = out_head_stride;
  p.rows = rows;
  p.heads = heads;
  const bool in_place = x == out && x_row_stride == out_row_stride && x_head_stride == out_head_stride;
  p.rope_chunk = offset / 8;
  p.first = in_place ? p.rope_chunk : 0;
  p.chunks = in_place ? mla::kRopeDim / 8 : width / 8;
  p.inverse = inverse != 0;
  p.positions = positions;
  // Blocks: a row's heads split until about eight blocks per SM exist, or
  // several rows to a block when one row's heads do not fill it.
  const int groups = mla::kRopeThreads / p.chunks;
  p.rows_per_block = groups / heads;
  int64_t grid;
  if (p.rows_per_block > 1) {
    p.head_blocks = 1;
    p.heads_per_block = heads;
    grid = (static_cast<int64_t>(rows) + p.rows_per_block - 1) / p.rows_per_block;
  } else {
    p.rows_per_block = 1;
    const int most = (heads + groups - 1) / groups;
    int64_t split = (int64_t(8) * ds->sms + rows - 1) / rows;
    if (split > most) split = most;
    p.heads_per_block = (most + static_cast<int>(split) - 1) / static_cast<int>(split) * groups;
    p.head_blocks = (heads + p.heads_per_block - 1) / p.heads_per_block;
    grid = static_cast<int64_t>(rows) * p.head_blocks;
  }
  if (grid > 0x7fffffff) return MLA_ERR_SHAPE;
  const mla::RopeTable tab = rope_table(*table);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tab.layout == MLA_ROPE_HALF)
    mla::rope_kernel<true><<<static_cast<unsigned>(grid), mla::kRopeThreads, 0, st>>>(tab, p);
  else
    mla::rope_kernel<false><<<static_cast<unsigned>(grid), mla::kRopeThreads, 0, st>>>(tab, p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_cache_append(const mla_rope_table* table, const void* kv_a, long long kv_a_row_stride,
                     const void* norm_weight, int weight_is_f32, float eps, const int32_t* positions,
                     const int32_t* slots, int rows, void* kv_cache, void* k_pe_cache, long long cache_rows,
                     mla_stream_t stream) {
  if (table == nullptr) return MLA_ERR_NULL;
  if (table->layout != MLA_ROPE_INTERLEAVED && table->layout != MLA_ROPE_HALF) return MLA_ERR_UNSUPPORTED;
  if (rows < 0 || cache_rows < 0 || kv_a_row_stride % 8 != 0 || kv_a_row_stride < kL + kDr) return MLA_ERR_SHAPE;
  if (!(eps >= 0.f) || !std::isfinite(eps) || (weight_is_f32 != 0 && weight_is_f32 != 1)) return MLA_ERR_SHAPE;
  if (rows == 0 || cache_rows == 0) return MLA_OK;
  if (!kv_a || !norm_weight || !positions || !kv_cache || !k_pe_cache) return MLA_ERR_NULL;
  if (!aligned16(kv_a) || !aligned16(norm_weight) || !aligned16(kv_cache) || !aligned16(k_pe_cache) ||
      ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 3u))
    return MLA_ERR_ALIGN;
  DeviceState* ds = nullptr;
  const int rc = device_state(&ds);
  if (rc != MLA_OK) return rc;
  mla::AppendParams p;
  p.kv_a = static_cast<const __nv_bfloat16*>(kv_a);
  p.kv_row = kv_a_row_stride;
  p.weight = norm_weight;
  p.weight_f32 = weight_is_f32 != 0;
  p.eps = eps;
  p.positions = positions;
  p.slots = slots;
  p.kv = static_cast<__nv_bfloat16*>(kv_cache);
  p.pe = static_cast<__nv_bfloat16*>(k_pe_cache);
  p.rows = rows;
  p.cache_rows = cache_rows;
  const mla::RopeTable tab = rope_table(*table);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = (static_cast<unsigned>(rows) + 3) / 4;
  if (tab.layout == MLA_ROPE_HALF)
    mla::cache_append_kernel<true><<<grid, 128, 0, st>>>(tab, p);
  else
    mla::cache_append_kernel<false><<<grid, 128, 0, st>>>(tab, p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_tree_decode(const mla_dims* dims, const mla_pages* pages, const void* q, const void* kv_cache,
                    const void* k_pe_cache, const int32_t* block_table, const int32_t* cache_len,
                    const int32_t* n_nodes, const int32_t* parents, const void* W_kvb, const float* W_kvb_scale,
                    const void* W_o, const float* W_o_scale, float scale, void* out, void* workspace,
                    size_t ws_bytes, mla_stream_t stream) {
  DeviceState* ds = nullptr;
  WsLayout lay;
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (dims->T > MLA_MAX_TREE) return MLA_ERR_SHAPE;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  if (static_cast<int64_t>(dims->B) * dims->T * dims->H > kMaxQueryRows) return MLA_ERR_SHAPE;
  if ((rc = check_pages(pages, true)) != MLA_OK) return rc;
  if (pages->layers != 1 || pages->num_pages < 1) return MLA_ERR_SHAPE;
  if (!q || !kv_cache || !k_pe_cache || !block_table || !cache_len || !W_kvb || !W_o || !out ||
      !fp8_scales_ok(dims, W_kvb_scale) || !fp8_scales_ok(dims, W_o_scale))
    return MLA_ERR_NULL;
  if (!std::isfinite(scale) || !(scale > 0.f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(k_pe_cache) || !aligned16(W_kvb) || !aligned16(W_o) ||
      !aligned16(out) || !aligned16(W_kvb_scale) || !aligned16(W_o_scale) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(cache_len) |
        reinterpret_cast<uintptr_t>(n_nodes) | reinterpret_cast<uintptr_t>(parents)) & 3u))
    return MLA_ERR_ALIGN;
  // A selection cannot be passed, so a model that sets one would get dense attention.
  if (dims->act != MLA_ACT_BF16 || dims->topk != 0) return MLA_ERR_UNSUPPORTED;
  rc = begin_call(dims, MLA_ENTRY_TREE_DECODE, false, workspace, ws_bytes, &ds, &lay);
  if (rc != MLA_OK) return rc;
  return run_tree_decode(ds, *dims, *pages, lay, workspace, q, kv_cache, k_pe_cache, block_table, cache_len, n_nodes,
                         parents, W_kvb, W_kvb_scale, W_o, W_o_scale, scale, out,
                         reinterpret_cast<cudaStream_t>(stream));
}

int mla_cache_compact(const mla_pages* pages, void* kv_cache, void* k_pe_cache, const int32_t* block_table,
                      const int32_t* cache_len, const int32_t* accepted, const int32_t* n_accepted, int B, int width,
                      mla_stream_t stream) {
  int rc = check_pages(pages, true);
  if (rc != MLA_OK) return rc;
  if (B < 0 || width < 0 || width > MLA_MAX_TREE) return MLA_ERR_SHAPE;
  if (B == 0 || width == 0 || pages->num_pages == 0) return MLA_OK;
  if (!kv_cache || !k_pe_cache || !block_table || !cache_len || !accepted || !n_accepted) return MLA_ERR_NULL;
  if (!aligned16(kv_cache) || !aligned16(k_pe_cache) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(cache_len) |
        reinterpret_cast<uintptr_t>(accepted) | reinterpret_cast<uintptr_t>(n_accepted)) & 3u))
    return MLA_ERR_ALIGN;
  DeviceState* ds = nullptr;
  if ((rc = device_state(&ds)) != MLA_OK) return rc;
  mla::CompactParams p;
  p.kv = static_cast<uint4*>(kv_cache);
  p.pe = static_cast<uint4*>(k_pe_cache);
  p.num_pages = pages->num_pages;
  p.page_shift = log2_of(pages->page_size);
  p.table_width = pages->table_width;
  p.table = block_table;
  p.cache_len = cache_len;
  p.accepted = accepted;
  p.counts = n_accepted;
  p.width = width;
  p.err = ds->err;
  p.layers = pages->layers;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto launch = [&](auto kernel, int side, int layers) {
    const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>((pages->layers + layers - 1) / layers));
    kernel<<<grid, mla::kRowPieces * side, 0, st>>>(p);
  };
  // By the most rows that a sequence can accept: enough registers for them, and
  // as many layers as leave two or more blocks on an SM. 64 sequences, 60 layers,
  // this choice and the next best: up to 5 rows 6.5 us (two layers 7.2), up to
  // 16 rows 15.7 (four layers 16.6, one 18), up to 32 rows 27.3 (two layers
  // and eight rows side by side 28.4), 64 rows each 97.7 (two layers 99.6).
  if (width <= 8)
    launch(mla::cache_compact_kernel<4, 2, 4>, 4, 4);
  else if (width <= 16)
    launch(mla::cache_compact_kernel<4, 4, 2>, 4, 2);
  else if (width <= 32)
    launch(mla::cache_compact_kernel<4, 8, 1>, 4, 1);
  else
    launch(mla::cache_compact_kernel<8, 8, 1>, 8, 1);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_cache_copy_pages(const mla_pages* pages, void* kv_cache, void* k_pe_cache, const int32_t* src,
                         const int32_t* dst, int n, mla_stream_t stream) {
  int rc = check_pages(pages, false);
  if (rc != MLA_OK) return rc;
  if (n < 0) return MLA_ERR_SHAPE;
  if (n == 0) return MLA_OK;
  if (!kv_cache || !k_pe_cache || !src || !dst) return MLA_ERR_NULL;
  if (!aligned16(kv_cache) || !aligned16(k_pe_cache)) return MLA_ERR_ALIGN;
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= pages->num_pages || dst[i] < 0 || dst[i] >= pages->num_pages) return MLA_ERR_SHAPE;
  // No destination twice, and none that another pair reads: the destinations in a
  // table with open addressing, at most half full, so that the check grows with
  // the list and not with the pool: 65 pairs of 2^20 pages 1.5 us, with one mark per
  // page 155; 64 pairs compared with one another took 1.5, too.
  if (n > pages->num_pages) return MLA_ERR_SHAPE;
  int bits = 1;
  while ((int64_t(1) << bits) < int64_t(2) * n) ++bits;
  const size_t slots = size_t(1) << bits;
  int few[128];
  int* const pair_at = slots <= 128 ? few : new (std::nothrow) int[slots];
  if (pair_at == nullptr) return MLA_ERR_CUDA;
  for (size_t i = 0; i < slots; ++i) pair_at[i] = -1;
  // Where page `v` is, or the free slot where it would be.
  auto find = [&](int v) -> int& {
    size_t at = (static_cast<uint32_t>(v) * 2654435769u) >> (32 - bits);
    while (pair_at[at] >= 0 && dst[pair_at[at]] != v) at = (at + 1) & (slots - 1);
    return pair_at[at];
  };
  bool ok = true;
  for (int i = 0; i < n && ok; ++i) {
    int& at = find(dst[i]);
    ok = at < 0;
    at = i;
  }
  for (int i = 0; i < n && ok; ++i) {
    const int at = find(src[i]);
    ok = at < 0 || at == i;
  }
  if (pair_at != few) delete[] pair_at;
  if (!ok) return MLA_ERR_SHAPE;
  DeviceState* ds = nullptr;
  if ((rc = device_state(&ds)) != MLA_OK) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int per = mla::kCopyThreads * mla::kCopyPer;
  const unsigned pieces = static_cast<unsigned>((int64_t(pages->page_size) * mla::kRowPieces + per - 1) / per);
  mla::PagePairs pp;
  for (int i = 0; i < n;) {
    int k = 0;
    for (; i < n && k < mla::kCopyPairs; ++i) {
      if (src[i] == dst[i]) continue;
      pp.src[k] = src[i];
      pp.dst[k] = dst[i];
      ++k;
    }
    if (k == 0) break;
    mla::cache_copy_kernel<<<dim3(pieces, static_cast<unsigned>(k), static_cast<unsigned>(pages->layers)),
                             mla::kCopyThreads, 0, st>>>(pp, static_cast<uint4*>(kv_cache),
                                                         static_cast<uint4*>(k_pe_cache), pages->num_pages,
                                                         pages->page_size);
    if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

const char* mla_status_str(int status) {
  switch (status) {
    case MLA_OK: return "ok";
    case MLA_ERR_NULL: return "a required pointer is NULL";
    case MLA_ERR_SHAPE: return "a size is out of range";
    case MLA_ERR_UNSUPPORTED: return "unsupported head geometry, weight type or device";
    case MLA_ERR_WORKSPACE: return "workspace missing or too small";
    case MLA_ERR_CUDA: return "a CUDA call or kernel launch failed";
    case MLA_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case MLA_ERR_DEVICE: return "a kernel recorded a device-side error";
    case MLA_ERR_TOO_LARGE: return "problem needs more scratch than the built-in MLA_STATIC_SCRATCH_BYTES";
    default: return "unknown status";
  }
}

int mla_device_status(mla_stream_t stream, int* device_error) {
  if (device_error == nullptr) return MLA_ERR_NULL;
  DeviceState* ds = nullptr;
  int rc = device_state(&ds);
  if (rc != MLA_OK) return rc;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, ds->err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return MLA_ERR_CUDA;
  if (v != 0 && cudaMemset(ds->err, 0, sizeof(int)) != cudaSuccess) return MLA_ERR_CUDA;
  *device_error = v;
  return MLA_OK;
}

int mla_set_e4m3_weight_conversion(int onchip) {
  if (onchip != 0 && onchip != 1) return MLA_ERR_SHAPE;
  g_e4m3_onchip = onchip;
  return MLA_OK;
}

int mla_set_wait_timeout_ns(unsigned long long ns) {
  const unsigned long long v = ns == 0 ? mla::kWaitTimeoutNs : ns;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaMemcpyToSymbol(mla::g_mla_wait_timeout_ns, &v, sizeof v) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_test_withhold_attention_loads(int on) {
  if (on < 0 || on > kWithholdFewRows) return MLA_ERR_SHAPE;
  const int v = on == kWithholdDense ? 1 : 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  if (cudaMemcpyToSymbol(mla::g_mla_withhold_attn_loads, &v, sizeof v) != cudaSuccess) return MLA_ERR_CUDA;
  g_withhold = on;
  return MLA_OK;
}

int mla_test_wo_split_plan(int tiles, int pairs, int num_kb, int* tail, int* split) {
  if (tail == nullptr || split == nullptr) return MLA_ERR_NULL;
  if (tiles < 0 || pairs < 0 || num_kb < 0) return MLA_ERR_SHAPE;
  float dummy = 0.f;  // any non-null workspace pointer: the plan only tests it for null
  const mla::GemmSplit sk = wo_split_plan(tiles, pairs, num_kb, &dummy);
  *tail = sk.tail;
  *split = sk.split;
  return MLA_OK;
}

int mla_profile_begin(void) {
  for (auto& r : t_prof.recs) {
    t_prof.pool.push_back(r.start);
    t_prof.pool.push_back(r.stop);
  }
  t_prof.recs.clear();
  t_prof.on = true;
  return MLA_OK;
}

int mla_profile_end(float* ms_total, int* launches) {
  if (ms_total == nullptr || launches == nullptr) return MLA_ERR_NULL;
  for (int i = 0; i < MLA_PROFILE_CLASSES; ++i) {
    ms_total[i] = 0.f;
    launches[i] = 0;
  }
  int rc = MLA_OK;
  for (auto& r : t_prof.recs) {
    float ms = 0.f;
    if (cudaEventSynchronize(r.stop) != cudaSuccess || cudaEventElapsedTime(&ms, r.start, r.stop) != cudaSuccess) {
      rc = MLA_ERR_CUDA;
      continue;
    }
    ms_total[r.cls] += ms;
    launches[r.cls] += 1;
  }
  for (auto& r : t_prof.recs) {
    t_prof.pool.push_back(r.start);
    t_prof.pool.push_back(r.stop);
  }
  t_prof.recs.clear();
  t_prof.on = false;
  return rc;
}

}  // extern "C"

// ------------------------------------------------------------------ built-in scratch entry point

// Scratch of mla_attend_static for callers that cannot allocate device
// memory. The module holds it on every GPU that loads the library.
__device__ __align__(256) uint8_t g_mla_static_scratch[MLA_STATIC_SCRATCH_BYTES];

namespace {

std::mutex g_static_mutex;
std::vector<uint8_t*> g_static_scratch;  // device address of the array, per device (NULL: not looked up)

// Device address of g_mla_static_scratch on the current device, looked up
// once per device. In host code the array's name is only a host-side
// stand-in, so kernels must be given this address instead.
int static_scratch(uint8_t** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_static_mutex);
  if (static_cast<int>(g_static_scratch.size()) <= dev) g_static_scratch.resize(dev + 1, nullptr);
  if (g_static_scratch[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_mla_static_scratch) != cudaSuccess || p == nullptr) return MLA_ERR_CUDA;
    g_static_scratch[dev] = static_cast<uint8_t*>(p);
  }
  *out = g_static_scratch[dev];
  return MLA_OK;
}

}  // namespace

extern "C" int mla_attend_static(const mla_dims* dims, const void* q, const void* kv_latent, const void* k_pe,
                                 const void* W_kvb, const float* W_kvb_scale, const int32_t* topk_idx, float scale,
                                 void* attn_out, mla_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (static_cast<int64_t>(dims->B) * dims->T == 0) return MLA_OK;
  if (!q || !kv_latent || !k_pe || !W_kvb || !attn_out || !fp8_scales_ok(dims, W_kvb_scale)) return MLA_ERR_NULL;
  if (topk_idx != nullptr && dims->topk < 1) return MLA_ERR_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv_latent) || !aligned16(k_pe) || !aligned16(W_kvb) || !aligned16(attn_out) ||
      !aligned16(W_kvb_scale) || !aligned16(topk_idx))
    return MLA_ERR_ALIGN;
  const WsLayout lay = ws_layout(*dims, MLA_ENTRY_ATTEND, topk_idx != nullptr);
  if (lay.total > MLA_STATIC_SCRATCH_BYTES) return MLA_ERR_TOO_LARGE;
  DeviceState* ds = nullptr;
  rc = device_state(&ds);
  if (rc != MLA_OK) return rc;
  uint8_t* scratch = nullptr;
  rc = static_scratch(&scratch);
  if (rc != MLA_OK) return rc;
  return run_attend(ds, *dims, lay, scratch, q, kv_latent, k_pe, W_kvb, W_kvb_scale, topk_idx, scale, attn_out,
                    reinterpret_cast<cudaStream_t>(stream));
}
