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
#include "prefix_attention.cuh"
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
  const int64_t warps2 = static_cast<int64_t>(p.n) * cdiv(heads, 2 * kGroups);
  // Few rows: one head a lane group, so that the latency of one load and one
  // store is all a call waits for; else two (32768 rows of 16 heads: one 89 us,
  // two 61, four 69).
  if (warps2 < h->num_sms * 16) {
    const int64_t warps = static_cast<int64_t>(p.n) * cdiv(heads, kGroups);
    launch_k(h->pdl, append_kv_kernel<D, 1>, dim3(static_cast<unsigned>((warps + 3) / 4)),
             dim3(128), 0, st, p);
  } else {
    const int64_t blocks = std::min<int64_t>((warps2 + 7) / 8, h->num_sms * 32);
    launch_k(h->pdl, append_kv_kernel<D, 2>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
             st, p);
  }
}

// Tokens of a CTA's slice of a row.
int sample_slice(int V) { return (cdiv(V, kSmpRanks) + 3) / 4 * 4; }

// Attention over a shared prefix: which kernel takes the prefix, how it is
// dealt, the splits of the requests' own keys, and the workspace.
struct PrefixPlan {
  int nt = 1, kt = 64;           // the prefix's kernel
  int tpt = 0, row_groups = 0, items = 0, tiles = 0, ctas = 0, max_segs = 0;
  int64_t run = 1;               // (item, tile) units of a CTA
  bool too_many = false;         // units, or own items, past 31 bits
  int chunk = 0, splits = 0, R = 0;
  size_t off_ml = 0, off_own = 0, off_own_ml = 0, total = 0;
};
PrefixPlan plan_prefix(const dflash_handle* h, int B, int q_len, int W, int prefix_pages) {
  const dflash_config& c = h->cfg;
  const int G = c.n_q_heads / c.n_kv_heads, Hkv = c.n_kv_heads, D = c.head_dim;
  PrefixPlan p;
  p.R = q_len * G;
  p.tpt = 128 / G;
  const int row_tiles = cdiv(B * q_len, p.tpt);
  if (prefix_pages > 0) {
    // One row tile: the prefix is a stream like the requests' own keys.  More:
    // two tiles share each key tile.
    p.nt = row_tiles > 1 ? 2 : 1;
    p.kt = p.nt == 2 ? 128 : 64;
    p.row_groups = cdiv(row_tiles, p.nt);
    p.items = Hkv * p.row_groups;
    p.tiles = cdiv(prefix_pages * 16, p.kt);
    const int64_t units = static_cast<int64_t>(p.items) * p.tiles;
    // One row tile leaves half of the CTAs that fit to the requests' own keys, and a
    // CTA at least 256 keys: its start costs as much as several tiles (16 single tokens
    // over 2048 shared keys, runs of two, four and eight tiles: 22.0, 19.3, 21.4 us).
    const int slots = h->num_sms;
    p.too_many = units > INT32_MAX;
    p.run = std::max<int64_t>(p.nt == 2 ? 2 : 4, (units + slots - 1) / slots);
    p.ctas = static_cast<int>((units + p.run - 1) / p.run);
    p.max_segs = static_cast<int>((p.run - 1) / p.tiles + 2);
  }
  const int own_keys = (W - prefix_pages) * 16;
  if (own_keys > 0) {
    // Two CTAs an SM if each has 2048 keys or less, for a CTA's start costs as much
    // as several tiles (32 requests of up to 2048 own keys in chunks of 448 against
    // 1792: 178 us against 176, with four times the parts); else shorter ones, down to
    // an eighth of an SM's share, which balance requests of different lengths (100 of
    // up to 8000: chunks of 8192 417 us, of 5440 378).
    const double per_sm = static_cast<double>(B) * Hkv * own_keys / h->num_sms;
    int chunk = static_cast<int>(std::ceil(std::max(per_sm / 8, std::min(per_sm / 2, 2048.0))));
    chunk = std::max(256, std::min(8192, (chunk + 63) / 64 * 64));
    p.chunk = chunk;
    p.splits = cdiv(own_keys, chunk);
    p.too_many |= static_cast<int64_t>(p.splits) * B * Hkv > INT32_MAX / 2;
  }
  const size_t pr = static_cast<size_t>(p.ctas) * p.max_segs * p.nt * 128;
  const size_t ow = static_cast<size_t>(p.splits) * B * Hkv * p.R;
  p.off_ml = align_up(pr * D * 4);
  p.off_own = p.off_ml + align_up(pr * 8);
  p.off_own_ml = p.off_own + align_up(ow * D * 4);
  p.total = p.off_own_ml + align_up(ow * 8) + kAlign;
  return p;
}

template <int D, int NT, int KT>
dflash_status launch_part(dflash_handle* h, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, const PartParams& p, int64_t ctas,
                          cudaStream_t st) {
  using C = PartCfg<D, NT, KT>;
  DF_CUDA(cudaFuncSetAttribute(attn_part_kernel<D, NT, KT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
  LaunchScope scope(h, DFLASH_KERNEL_PREFIX_ATTENTION, st);
  launch_k(h->pdl, attn_part_kernel<D, NT, KT>, dim3(static_cast<unsigned>(ctas)),
           dim3(C::kThreads), C::kSmem, st, tq, tk, tv, p);
  return DFLASH_OK;
}

// Query tokens [n_tok][Hq][D] in boxes of tpt tokens x G heads x 64 columns.
bool make_q_map(CUtensorMap* map, const void* q, int n_tok, int Hq, int D, int G, int tpt) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq),
                        static_cast<cuuint64_t>(n_tok)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hq) * D * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tpt)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
dflash_status run_prefix(dflash_handle* h, const PrefixPlan& pl, PartParams p, const void* q,
                         const void* kc, const void* vc, f16* o, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  const uint64_t rows = static_cast<uint64_t>(p.num_pages) * p.Hkv * 16;
  if (!make_q_map(&tq, q, p.n_tok, p.Hq, D, p.G, p.tpt) || !h->tmap(&tk, kc, rows, D, 16) ||
      !h->tmap(&tv, vc, rows, D, 16))
    return DFLASH_ERR_CUDA;
  dflash_status s = DFLASH_OK;
  PartParams own = p;
  if (pl.nt == 2) {
    s = launch_part<D, 2, 128>(h, tq, tk, tv, p, pl.ctas, st);
    own.prefix_ctas = 0;
  }
  // one CTA an item of own keys: CTAs that stayed and took several items in turn
  // balanced worse (16 single tokens over 2048 shared keys 36 us against 25)
  const int64_t ctas = own.prefix_ctas + static_cast<int64_t>(pl.splits) * p.B * p.Hkv;
  if (s == DFLASH_OK && ctas > 0) s = launch_part<D, 1, 64>(h, tq, tk, tv, own, ctas, st);
  if (s != DFLASH_OK) return s;
  LaunchScope scope(h, DFLASH_KERNEL_PREFIX_COMBINE, st);
  // a warp a kv group once those occupy the card, else a warp a head (tokens of 8
  // groups, whole calls: 16 21.4 and 18.0 us, 128 91 and 89, 256 63 and 66, 512 168
  // and 175, 1024 160 and 183)
  const int heads = static_cast<int64_t>(p.n_tok) * p.Hkv >= 10 * h->num_sms ? p.G : 1;
  const int64_t warps = static_cast<int64_t>(p.n_tok) * (p.Hq / heads);
  launch_k(h->pdl, attn_join_kernel<D>, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0,
           st, p, pl.nt, heads, o);
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

// Geometry of a prefix-attention call: OK or what is wrong with it.
dflash_status check_prefix(const dflash_handle* h, int B, int q_len, int W, int prefix_pages) {
  if (!h || B < 0 || q_len < 1 || W < 1 || prefix_pages < 0 || prefix_pages > W)
    return DFLASH_ERR_INVALID_ARG;
  const int G = h->cfg.n_q_heads / h->cfg.n_kv_heads;
  if (B > 65535 || q_len * static_cast<int64_t>(G) > 128 || W > (1 << 24))
    return DFLASH_ERR_UNSUPPORTED_SHAPE;
  return DFLASH_OK;
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

size_t dflash_prefix_attention_workspace_bytes(const dflash_handle* h, int B, int q_len,
                                               int max_pages_per_seq, int prefix_pages) {
  if (check_prefix(h, B, q_len, max_pages_per_seq, prefix_pages) != DFLASH_OK || B == 0) return 0;
  return plan_prefix(h, B, q_len, max_pages_per_seq, prefix_pages).total;
}

dflash_status dflash_prefix_attention(dflash_handle* h, const void* q, int q_len, int causal,
                                      const int32_t* seq_lens, const int32_t* block_table, int B,
                                      int max_pages_per_seq, int prefix_pages,
                                      const void* k_cache, const void* v_cache, int num_pages,
                                      void* o, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  const dflash_status s = check_prefix(h, B, q_len, max_pages_per_seq, prefix_pages);
  if (s != DFLASH_OK || B == 0) return s;
  if (!q || !seq_lens || !block_table || !k_cache || !v_cache || num_pages < 1 || !o ||
      !workspace || !aligned16(q) || !aligned16(o) || !aligned16(k_cache) || !aligned16(v_cache) ||
      reinterpret_cast<uintptr_t>(workspace) % kAlign)
    return DFLASH_ERR_INVALID_ARG;
  const dflash_config& c = h->cfg;
  if (static_cast<int64_t>(num_pages) * c.n_kv_heads * 16 > INT32_MAX)
    return DFLASH_ERR_UNSUPPORTED_SHAPE;   // rows of the pools' tensor maps
  const PrefixPlan pl = plan_prefix(h, B, q_len, max_pages_per_seq, prefix_pages);
  if (pl.too_many) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < pl.total) return DFLASH_ERR_WORKSPACE;
  DF_CUDA(use_device(h->device));
  PartParams p;
  p.B = B;
  p.q_len = q_len;
  p.n_tok = B * q_len;
  p.Hq = c.n_q_heads;
  p.Hkv = c.n_kv_heads;
  p.G = c.n_q_heads / c.n_kv_heads;
  p.tpt = pl.tpt;
  p.causal = causal ? 1 : 0;
  p.q = static_cast<const bf16*>(q);
  p.k_cache = static_cast<const bf16*>(k_cache);
  p.v_cache = static_cast<const bf16*>(v_cache);
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.W = max_pages_per_seq;
  p.num_pages = num_pages;
  p.prefix_keys = prefix_pages * 16;
  p.prefix_ctas = pl.ctas;
  p.prefix_items = pl.items;
  p.prefix_tiles = pl.tiles;
  p.prefix_run = static_cast<unsigned>(pl.run);
  p.row_groups = pl.row_groups;
  p.max_segs = pl.max_segs;
  p.prefix_o = at<float>(workspace, 0);
  p.prefix_ml = at<float2>(workspace, pl.off_ml);
  p.chunk_keys = pl.chunk;
  p.max_splits = pl.splits;
  p.R = pl.R;
  p.own_o = at<float>(workspace, pl.off_own);
  p.own_ml = at<float2>(workspace, pl.off_own_ml);
  p.scale_log2 =
      static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(c.head_dim)));
  p.err = h->dev_err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c.head_dim == 128 ? run_prefix<128>(h, pl, p, q, k_cache, v_cache,
                                             static_cast<f16*>(o), st)
                           : run_prefix<64>(h, pl, p, q, k_cache, v_cache, static_cast<f16*>(o),
                                            st);
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
  SampleParams p;
  p.logits = logits;
  p.ld = ld;
  p.rows = rows;
  p.V = V;
  p.slice = sample_slice(V);
  p.set = {temperature, top_k, top_p, min_p};
  p.u = u;
  p.tokens = tokens;
  p.probs = probs;
  p.err = device_error;
  launch_kc(pdl_default(), kSmpRanks, sample_kernel, dim3(kSmpRanks, rows), dim3(kSmpThreads),
            sizeof(SmpShared), st, p);
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
  VerifySampledParams p;
  p.drafts = drafts;
  p.logits = target_logits;
  p.ld = ld;
  p.B = B;
  p.K = K;
  p.V = V;
  p.slice = sample_slice(V);
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
  launch_k(pdl_default(), zero_words_kernel, dim3(std::min(cdiv(2 * B, 256), 64)), dim3(256), 0,
           st, p.done, 2 * B);
  launch_kc(pdl_default(), kSmpRanks, verify_sampled_kernel, dim3(kSmpRanks, B, K + 1),
            dim3(kSmpThreads), sizeof(SmpShared), st, p);
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
