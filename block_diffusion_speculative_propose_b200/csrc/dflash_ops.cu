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
#include "sampling.cuh"

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

// Cluster size and slice for a vocabulary: a CTA a slice of up to 8192 tokens,
// at most eight CTAs (the portable cluster size).
struct SamplePlan {
  int ranks = 1, slice = 0;
  size_t smem = 0;
};
SamplePlan plan_sample(int V) {
  SamplePlan p;
  while (p.ranks < kSmpMaxCluster && p.ranks * 8192 < V) p.ranks *= 2;
  p.slice = (cdiv(V, p.ranks) + 3) / 4 * 4;
  p.smem = smp_smem_bytes(p.slice);
  return p;
}

__global__ void zero_words_kernel(unsigned* p, int n) {
  pdl_trigger();
  pdl_wait();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) p[i] = 0;
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

dflash_status dflash_sample_tokens(const float* logits, int64_t ld, int rows, int V,
                                   const float* temperature, const int32_t* top_k,
                                   const float* top_p, const float* min_p, const float* u,
                                   int32_t* tokens, float* probs, unsigned* device_error,
                                   void* stream) {
  if (rows < 0 || V < 1) return DFLASH_ERR_INVALID_ARG;
  if (rows == 0) return DFLASH_OK;
  if (!logits || !u || !tokens || ld < V || reinterpret_cast<uintptr_t>(logits) % 4)
    return DFLASH_ERR_INVALID_ARG;
  if (V > kSmpMaxVocab || rows > 65535) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dflash_status s = set_device_for(st, tokens);
  if (s != DFLASH_OK) return s;
  const SamplePlan pl = plan_sample(V);
  SampleParams p;
  p.logits = logits;
  p.ld = ld;
  p.rows = rows;
  p.V = V;
  p.slice = pl.slice;
  p.set = {temperature, top_k, top_p, min_p};
  p.u = u;
  p.tokens = tokens;
  p.probs = probs;
  p.err = device_error;
  DF_CUDA(cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(pl.smem)));
  launch_kc(pdl_default(), pl.ranks, sample_kernel, dim3(pl.ranks, rows), dim3(kSmpThreads),
            pl.smem, st, p);
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

size_t dflash_verify_sampled_workspace_bytes(int B, int K) {
  if (B <= 0 || K < 0) return 0;
  return align_up(static_cast<size_t>(B) * (K + 3) * 4);
}

dflash_status dflash_verify_sampled(const int32_t* drafts, const float* target_logits, int64_t ld,
                                    int B, int K, int V, const float* temperature,
                                    const int32_t* top_k, const float* top_p, const float* min_p,
                                    const float* u_accept, const float* u_sample,
                                    int32_t* out_tokens, int32_t* num_accepted, int32_t* bonus,
                                    unsigned* device_error, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (B < 0 || K < 0 || V < 1 || K > 128) return DFLASH_ERR_INVALID_ARG;
  if (B == 0) return DFLASH_OK;
  if ((K > 0 && (!drafts || !u_accept)) || !target_logits || !u_sample || !out_tokens ||
      !num_accepted || !bonus || !workspace || ld < V ||
      reinterpret_cast<uintptr_t>(target_logits) % 4 || reinterpret_cast<uintptr_t>(workspace) % 4)
    return DFLASH_ERR_INVALID_ARG;
  if (V > kSmpMaxVocab || B > 65535) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < dflash_verify_sampled_workspace_bytes(B, K)) return DFLASH_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dflash_status s = set_device_for(st, out_tokens);
  if (s != DFLASH_OK) return s;
  const SamplePlan pl = plan_sample(V);
  VerifySampledParams p;
  p.drafts = drafts;
  p.logits = target_logits;
  p.ld = ld;
  p.B = B;
  p.K = K;
  p.V = V;
  p.slice = pl.slice;
  p.set = {temperature, top_k, top_p, min_p};
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.out = out_tokens;
  p.num_accepted = num_accepted;
  p.bonus = bonus;
  p.err = device_error;
  p.done = static_cast<unsigned*>(workspace);
  p.refused = p.done + B;
  p.row_token = static_cast<int32_t*>(workspace) + 2 * static_cast<int64_t>(B);
  DF_CUDA(cudaFuncSetAttribute(verify_sampled_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(pl.smem)));
  launch_k(pdl_default(), zero_words_kernel, dim3(std::min(cdiv(2 * B, 256), 64)), dim3(256), 0,
           st, p.done, 2 * B);
  launch_kc(pdl_default(), pl.ranks, verify_sampled_kernel, dim3(pl.ranks, B, K + 1),
            dim3(kSmpThreads), pl.smem, st, p);
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
