// handle.cuh — what every source file of the C ABI shares on the host: the
// handle, tensor-map construction, launch helpers and device selection.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <array>
#include <cstdlib>
#include <map>
#include <mutex>
#include <tuple>
#include <vector>

#include "dflash.h"
#include "dflash_device.cuh"

using namespace dflash;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t v, size_t a = kAlign) { return (v + a - 1) / a * a; }
int cdiv(int a, int b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// driver entry point for tensor-map encoding (no link-time libcuda dependency)
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D view of 16-bit elements (bf16, or fp16 when f16) [rows][cols] (row pitch
// cols * 2 bytes), box [box_rows][64], 128-byte swizzle.  Out-of-range box
// rows read as zeros.
bool make_tmap(CUtensorMap* map, const void* ptr, uint64_t rows, uint64_t cols,
               uint32_t box_rows, bool f16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(ptr), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------------------
// error helpers
// ---------------------------------------------------------------------------
#define DF_CUDA(expr)                                   \
  do {                                                  \
    if ((expr) != cudaSuccess) return DFLASH_ERR_CUDA;  \
  } while (0)

}  // namespace

// Programmatic dependent launch unless the environment sets DFLASH_PDL=0
// (read once per process).
inline bool pdl_default() {
  static const bool on = [] {
    const char* e = std::getenv("DFLASH_PDL");
    return !(e && e[0] == '0');
  }();
  return on;
}

// ---------------------------------------------------------------------------
// handle
// ---------------------------------------------------------------------------
struct dflash_handle {
  dflash_config cfg{};
  std::vector<int> target_layer_ids;
  int device = 0;
  int num_sms = 148;
  // aliased caller weights (embedding table and norm weights)
  const bf16 *hidden_norm_w = nullptr, *embed = nullptr, *final_norm_w = nullptr;
  std::vector<const bf16*> in_norm_w, post_norm_w, q_norm_w, k_norm_w;
  // GEMM weights: copies owned by the handle, in the tile-contiguous layout of
  // pack_tiles_kernel; the ones multiplied against fp16 operands are held as
  // fp16 (bf16 -> fp16 is exact in fp16's normal range)
  std::vector<f16*> wqkv, wgu, wo;  // [Wq; Wk; Wv], gate/up interleaved by 16 rows, Wo
  std::vector<bf16*> wdown;         // W_down (bf16: multiplied against the bf16 MLP hidden)
  bf16* fcw = nullptr;              // fc (bf16: multiplied against the bf16 target states)
  f16* wkv = nullptr;               // all layers' [Wk; Wv], [L * 2 * Hkv * D, H]
  f16* lm_head16 = nullptr;         // [vocab_count, H]: rows [vocab_start, +vocab_count)
  // vocabulary shard of the LM head (tensor-parallel proposal); the whole
  // vocabulary unless created by dflash_create_vocab_shard
  int vocab_start = 0, vocab_count = 0;
  // tensor-parallel shard (dflash_create_tp_shard): rank and group size; the
  // cfg above then holds this shard's head and MLP-feature counts
  int tp_rank = 0, tp_size = 1;
  bf16* knorm_all = nullptr;  // [L, D]
  float2* rope = nullptr;   // [max_position, D/2]
  unsigned* dev_err = nullptr;
  unsigned* counters = nullptr;
  // fp16 range of the weights stored in fp16 (checked by dflash_create)
  unsigned* range_stats = nullptr;
  float fp16_weight_absmax = 0.f;
  double fp16_subnormal_fraction = 0.0;
  double norm_output_bound = 0.0;
  std::mutex mu;
  std::map<std::tuple<const void*, uint64_t, uint64_t, uint32_t, bool>, CUtensorMap> tmaps;
  std::map<std::pair<const void*, int>, std::array<int, 9>> cluster_caps;
  // launch accounting and optional per-launch event profiling (diagnostics)
  unsigned long long launches = 0;
  bool prof_on = false;
  // hot-path kernels are launched with programmatic dependent launch (the
  // environment variable DFLASH_PDL=0 turns it off)
  bool pdl = pdl_default();
  // few-row gate/up + down as one chain launch: opt-in (DFLASH_CHAIN=1 when the
  // handle is created).  Measured on the batch-1 Qwen3-8B-shaped step it is
  // 1-2% slower than two launches, whose down GEMM already prefetches on the
  // SMs gate/up leaves free and reduces through clusters.
  bool chain = [] {
    const char* e = std::getenv("DFLASH_CHAIN");
    return e && e[0] == '1';
  }();
  // cluster-combined attention splits for few requests: opt-in
  // (DFLASH_ATTN_CLUSTER=1 when the handle is created)
  bool attn_cluster = [] {
    const char* e = std::getenv("DFLASH_ATTN_CLUSTER");
    return e && e[0] == '1';
  }();
  // K/V ring depth of the 64-key attention kernel forced by DFLASH_ATTN_STAGES
  // (2 or 6) when the handle is created; 0 lets the planner decide
  int attn_ring = [] {
    const char* e = std::getenv("DFLASH_ATTN_STAGES");
    return e ? std::atoi(e) : 0;
  }();
  // six-deep-ring attention as persistent CTAs: opt-in (DFLASH_ATTN_PERSIST=1
  // when the handle is created)
  bool attn_persist = [] {
    const char* e = std::getenv("DFLASH_ATTN_PERSIST");
    return e && e[0] == '1';
  }();
  // keys per tile of the two-CTA-per-SM head_dim-128 kernel (DFLASH_ATTN_TILE
  // = 32 or 64 when the handle is created; 64 otherwise: measured at 128
  // requests x 8k-32k keys, 64-key tiles stream 4.2 TB/s, 32-key ones 3.7)
  int attn_tile = [] {
    const char* e = std::getenv("DFLASH_ATTN_TILE");
    return (e && std::atoi(e) == 32) ? 32 : 64;
  }();
  // whole-tile GEMMs over several 128-row M tiles run on CTA pairs (one MMA of
  // 256 x 256 over two SMs, gemm_pair.cuh) unless DFLASH_GEMM_PAIR=0 when the
  // handle is created
  bool gemm_pair = [] {
    const char* e = std::getenv("DFLASH_GEMM_PAIR");
    return !(e && e[0] == '0');
  }();
  // few wide pair tiles with a long K split over two pairs (a cluster of four)
  // unless DFLASH_GEMM_SPLIT=0 when the handle is created
  bool gemm_split = [] {
    const char* e = std::getenv("DFLASH_GEMM_SPLIT");
    return !(e && e[0] == '0');
  }();
  // two-CTA clusters of each pair-GEMM instantiation that can be resident at
  // once (occupancy query, per kernel)
  std::map<const void*, int> pair_clusters;
  std::vector<cudaEvent_t> prof_events;
  size_t prof_next = 0;
  std::vector<int> prof_kind;

  bool tmap(CUtensorMap* out, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows,
            bool f16 = false) {
    std::lock_guard<std::mutex> lk(mu);
    auto key = std::make_tuple(ptr, rows, cols, box_rows, f16);
    auto it = tmaps.find(key);
    if (it != tmaps.end()) {
      *out = it->second;
      return true;
    }
    if (tmaps.size() > 8192) tmaps.clear();
    if (!make_tmap(out, ptr, rows, cols, box_rows, f16)) return false;
    tmaps.emplace(key, *out);
    return true;
  }
};

namespace {

// Counts every kernel launch a handle's call makes and, while profiling is on,
// brackets it with a pair of events recorded on the launching stream.
struct LaunchScope {
  dflash_handle* h;
  cudaStream_t st;
  cudaEvent_t stop = nullptr;
  LaunchScope(dflash_handle* h_, int kind, cudaStream_t st_) : h(h_), st(st_) {
    ++h->launches;
    if (h->prof_on && h->prof_next + 2 <= h->prof_events.size()) {
      cudaEvent_t a = h->prof_events[h->prof_next];
      stop = h->prof_events[h->prof_next + 1];
      h->prof_next += 2;
      h->prof_kind.push_back(kind);
      cudaEventRecord(a, st);
    }
  }
  ~LaunchScope() {
    if (stop) cudaEventRecord(stop, st);
  }
};

// Launch of a hot-path kernel; with `pdl` the launch may overlap the tail of
// the previous kernel in the stream (every such kernel calls pdl_wait() before
// it touches memory that an earlier kernel writes or a later one overwrites).
// `cluster` > 1 launches thread-block clusters of that many CTAs along x.
template <typename... KArgs, typename... Args>
void launch_kc(bool pdl, int cluster, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
               cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
void launch_k(bool pdl, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
              cudaStream_t st, Args&&... args) {
  launch_kc(pdl, 1, kern, grid, block, smem, st, std::forward<Args>(args)...);
}

template <class T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + off);
}

// Makes `dev` current for this library's runtime (a no-op when it already is,
// so calls stay cheap and legal inside stream capture).
cudaError_t use_device(int dev) {
  int cur = -1;
  if (cudaGetDevice(&cur) == cudaSuccess && cur == dev) return cudaSuccess;
  return cudaSetDevice(dev);
}

// Handle-free calls run on the device of their stream (or, on the legacy
// default stream, of their output buffer).
// Under stream capture the device is not queried (a stream query would
// invalidate a global-mode capture); the current device is used as is.
dflash_status set_device_for(cudaStream_t st, const void* p) {
  int dev = -1;
  if (st != nullptr) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) {
      cudaGetLastError();
      return DFLASH_ERR_INVALID_ARG;
    }
    if (cs != cudaStreamCaptureStatusNone) return DFLASH_OK;
    if (cudaStreamGetDevice(st, &dev) != cudaSuccess) {
      cudaGetLastError();
      return DFLASH_ERR_INVALID_ARG;
    }
  } else {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess || a.type != cudaMemoryTypeDevice) {
      cudaGetLastError();
      return DFLASH_ERR_INVALID_ARG;
    }
    dev = a.device;
  }
  DF_CUDA(use_device(dev));
  return DFLASH_OK;
}

}  // namespace
