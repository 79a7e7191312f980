// dflash_ops.cu — the C ABI's operators around a draft block that the caller
// composes itself: appending to the paged caches, attention over a shared
// prefix, sampling and sampled verification.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "append_kv.cuh"
#include "dflash.h"
#include "handle.cuh"

namespace dflash {
// The wait limit that this file's kernels read (see dflash_set_wait_limit).
cudaError_t set_ops_wait_limit(long long cycles) {
  return cudaMemcpyToSymbol(g_wait_limit_cycles, &cycles, sizeof(cycles));
}
}  // namespace dflash

namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int D>
void launch_append(dflash_handle* h, const AppendParams& p, cudaStream_t st) {
  LaunchScope scope(h, DFLASH_KERNEL_APPEND_KV, st);
  const int heads = 2 * p.Hkv + (p.q ? p.Hq : 0);
  constexpr int kGroups = 512 / D;
  const int64_t warps4 = static_cast<int64_t>(p.n) * cdiv(heads, 4 * kGroups);
  // Few rows: one head a lane group, so that the latency of one load and one
  // store is all a call waits for; else four.
  if (warps4 < h->num_sms * 8) {
    const int64_t warps = static_cast<int64_t>(p.n) * cdiv(heads, kGroups);
    launch_k(h->pdl, append_kv_kernel<D, 1>, dim3(static_cast<unsigned>((warps + 3) / 4)),
             dim3(128), 0, st, p);
  } else {
    const int64_t blocks = std::min<int64_t>((warps4 + 7) / 8, h->num_sms * 32);
    launch_k(h->pdl, append_kv_kernel<D, 4>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
             st, p);
  }
}

}  // namespace

extern "C" {

dflash_status dflash_append_kv(dflash_handle* h, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, const void* k_norm_w, const void* q,
                               int64_t q_stride, const void* q_norm_w, void* q_out,
                               const int64_t* positions, const int64_t* slot_mapping, int n,
                               void* k_cache, void* v_cache, int num_pages, void* stream) {
  if (!h || n < 0) return DFLASH_ERR_INVALID_ARG;
  if (n == 0) return DFLASH_OK;
  if (!k || !v || !positions || !slot_mapping || !k_cache || !v_cache || num_pages < 1 ||
      (q == nullptr) != (q_out == nullptr) || (q_norm_w && !q))
    return DFLASH_ERR_INVALID_ARG;
  const dflash_config& c = h->cfg;
  const int64_t kv = static_cast<int64_t>(c.n_kv_heads) * c.head_dim;
  const int64_t qd = static_cast<int64_t>(c.n_q_heads) * c.head_dim;
  if (k_stride < kv || v_stride < kv || (q && q_stride < qd) || k_stride % 8 || v_stride % 8 ||
      (q && q_stride % 8))
    return DFLASH_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) ||
      !aligned16(k_norm_w) || !aligned16(q_norm_w) || !aligned16(k_cache) || !aligned16(v_cache))
    return DFLASH_ERR_INVALID_ARG;
  // in place only where every element is read and written by the same lane
  if (q && q == q_out && q_stride != qd) return DFLASH_ERR_INVALID_ARG;
  DF_CUDA(use_device(h->device));
  AppendParams p;
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.q = static_cast<const bf16*>(q);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.k_norm = static_cast<const bf16*>(k_norm_w);
  p.q_norm = static_cast<const bf16*>(q_norm_w);
  p.positions = positions;
  p.slots = slot_mapping;
  p.n = n;
  p.num_pages = num_pages;
  p.Hq = c.n_q_heads;
  p.Hkv = c.n_kv_heads;
  p.page_size = c.page_size;
  p.max_position = c.max_position;
  p.eps = c.rms_eps;
  p.rope = h->rope;
  p.k_cache = static_cast<bf16*>(k_cache);
  p.v_cache = static_cast<bf16*>(v_cache);
  p.q_out = static_cast<bf16*>(q_out);
  p.err = h->dev_err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c.head_dim == 128) launch_append<128>(h, p, st);
  else launch_append<64>(h, p, st);
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
