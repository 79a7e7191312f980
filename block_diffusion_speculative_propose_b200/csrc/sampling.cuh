// sampling.cuh — a draw from the filtered distribution of a row of logits, and
// the acceptance of a greedy draft against it.
//
// For a row x (NaN counts as -inf), its largest entry m and a temperature T > 0
// every token weighs w = exp((x - m) / T).  In the order of falling x (ties:
// lower id first) a prefix of the tokens is kept: the first top_k; those of
// them with w >= min_p; and of these the shortest prefix whose weight reaches
// top_p of theirs.  The drawn token is the first in vocabulary order whose
// running sum of kept weights passes u times their sum.
//
// Numbers.  A draw near a border must not depend on rounding, nor on the order
// in which parts are added: each weight is computed in 64 bits and rounded once
// to an integer W = rint(w 2^44); every sum is a sum of integers, exact in any
// order (V <= 2^18.6 weights of at most 2^44).  Tokens below 2^-45 of the
// largest weigh nothing.
//
// Layout.  A row is held by a cluster: each of its CTAs copies one slice of the
// row to shared memory, so the logits are read from memory once however many
// passes the filters need; what the CTAs have to tell one another goes through
// distributed shared memory.
#pragma once

#include "dflash_device.cuh"

namespace dflash {

constexpr int kSmpThreads = 512;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpMaxCluster = 8;
constexpr int kSmpBins = 1024;        // linear bins of x below the maximum
constexpr int kSmpRadix = 2048;       // bins of a radix level (11 bits)
constexpr int kSmpList = 1024;        // candidates that one CTA sorts
constexpr int kSmpOneBits = 44;       // W of the largest weight: 2^44
constexpr float kSmpReach = 31.9f;    // 46 ln 2: tokens further below weigh nothing
constexpr int kSmpMaxVocab = 393216;  // 8 slices of 192 KiB

typedef unsigned long long u64;

struct SampleSettings {
  const float* temperature;   // one entry per row (or request); null: 1
  const int32_t* top_k;       // null or <= 0: off
  const float* top_p;         // null: 1
  const float* min_p;         // null: 0
};

// What the CTAs of a cluster show one another; every field is written once a
// row, so a barrier between the writing and the reading is all it needs.
struct SmpShared {
  double tab[32];                    // 2^(j / 32)
  u64 warp_a[kSmpWarps];             // block-wide sums
  u64 bcast[4];
  u64 top_key;                       // phase A: largest (value, id)
  float low;                         // phase A: smallest finite value
  u64 mass_all;                      // weight of the whole slice
  u64 ties[2];                       // ties of the border value (two searches)
  u64 border[2];                     // the border key (two searches)
  u64 kept, draft_w;                 // the slice's kept weight, the draft's weight
  unsigned n_local;
  unsigned first_bad;
  unsigned cnt[kSmpRadix];           // histogram: tokens
  union {
    unsigned mass[2][kSmpRadix];     // histogram: low and high words of weights
    struct {
      u64 list[kSmpList];            // rank 0: the candidates' keys
      u64 w[kSmpList];
    };
  };
};

__host__ __device__ constexpr size_t smp_smem_bytes(int slice) {
  return sizeof(SmpShared) + static_cast<size_t>(slice) * 4 + 16;
}

__device__ __forceinline__ uint32_t smp_order(float x) {   // orders like x (no NaN, no -0)
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float smp_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ u64 smp_key(float x, uint32_t id) {
  return (static_cast<u64>(smp_order(x)) << 32) | (0xffffffffu - id);
}
__device__ __forceinline__ uint32_t smp_id(u64 key) {
  return 0xffffffffu - static_cast<uint32_t>(key);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ u64 ld_peer_u64(const void* p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_peer_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer_u64(void* p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_addr(p, rank)), "l"(v) : "memory");
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan_u64(u64 v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// One row as the cluster's threads see it.
struct SmpRow {
  SmpShared* sh;
  const float* x;        // this CTA's slice (NaN as -inf, -0 as +0)
  int len, begin;        // its length and first id
  int rank, ranks;
  float m;               // the row's largest value
  double c;              // log2(e) / T
  u64 w_min;             // min_p as a weight
};

// W of value x: 0 where it is filtered by min_p or weighs nothing.  With
// t = (x - m) log2(e) / T = n/32 + f, 2^t = 2^(n >> 5) 2^((n & 31) / 32) 2^f,
// |f| <= 1/64: five terms of 2^f's Taylor series leave 2^-48 relative.
__device__ __forceinline__ u64 smp_weight(const SmpRow& r, float x) {
  const double d = x == r.m ? 0.0 : static_cast<double>(x) - static_cast<double>(r.m);
  const double t = d * r.c;
  if (!(t >= -46.0)) return 0ull;
  const double magic = 6755399441055744.0;   // 1.5 2^52: the sum's low bits are rint(32 t)
  const double s = __fma_rn(t, 32.0, magic);
  const int n = __double2loint(s);
  const double f = __fma_rn(t, 32.0, magic - s);
  const double a = 0.6931471805599453 / 32.0;   // ln 2 / 32
  double p = a * a * a * a * a / 120.0;
  p = __fma_rn(p, f, a * a * a * a / 24.0);
  p = __fma_rn(p, f, a * a * a / 6.0);
  p = __fma_rn(p, f, a * a / 2.0);
  p = __fma_rn(p, f, a);
  p = __fma_rn(p, f, 1.0);
  p *= r.sh->tab[n & 31];
  // times 2^((n >> 5) + 44), then the integer nearest (n >> 5 >= -46: normal)
  const double v = __hiloint2double(__double2hiint(p) + (((n >> 5) + kSmpOneBits) << 20),
                                    __double2loint(p));
  const u64 w = static_cast<u64>(__double_as_longlong(v + 4503599627370496.0)) & 0xfffffffffffffull;
  return w < r.w_min ? 0ull : w;
}

// Block-wide sum; every thread gets it.
__device__ __forceinline__ u64 smp_block_sum(SmpShared* sh, u64 v) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum_u64(v);
  __syncthreads();
  if (lane == 0) sh->warp_a[warp] = v;
  __syncthreads();
  return warp_sum_u64(lane < kSmpWarps ? sh->warp_a[lane] : 0ull);
}
// Block-wide inclusive scan of one value a thread (in thread order).
__device__ __forceinline__ u64 smp_block_scan(SmpShared* sh, u64 v) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_scan_u64(v, lane);
  __syncthreads();
  if (lane == 31) sh->warp_a[warp] = v;
  __syncthreads();
  const u64 before = warp_sum_u64(lane < warp ? sh->warp_a[lane] : 0ull);
  return v + before;
}

// Falling bitonic sort of a[0..n), n a power of two.
__device__ __forceinline__ void smp_sort(u64* a, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += kSmpThreads) {
        const int lo = 2 * i - (i & (j - 1));
        const u64 p = a[lo], q = a[lo + j];
        if ((p < q) == ((lo & k) == 0)) {
          a[lo] = q;
          a[lo + j] = p;
        }
      }
    }
  __syncthreads();
}

// The border of a kept prefix among the tokens with key >= floor_key: the key
// of the `want`-th of them (by_mass false), or of the first at which their
// running weight reaches top_p of all of theirs.  Every CTA of the cluster
// takes part and gets the same answer.  Three radix levels find the value, then
// the ties at it are counted in vocabulary order; `which` (0, 1) separates the
// shared fields of a row's two searches.
__device__ u64 smp_border(const SmpRow& r, bool by_mass, u64 floor_key, u64 want, double top_p,
                          int which) {
  SmpShared* sh = r.sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t prefix = 0;
  u64 base = 0;             // tokens, or weight, above the current prefix
  double goal = 0.0;        // by mass: the weight to reach
  u64 bin_cnt = 0;
  constexpr int kPer = kSmpRadix / kSmpThreads;
  for (int level = 0; level < 3; ++level) {
    const int bits = level == 2 ? 10 : 11;
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
    for (int i = tid; i < kSmpRadix; i += kSmpThreads) {
      sh->cnt[i] = 0;
      sh->mass[0][i] = 0;
      sh->mass[1][i] = 0;
    }
    __syncthreads();
    for (int i = tid; i < r.len; i += kSmpThreads) {
      const float x = r.x[i];
      const u64 key = smp_key(x, r.begin + i);
      const uint32_t o = static_cast<uint32_t>(key >> 32);
      if (key < floor_key || (level > 0 && (o >> (shift + bits)) != prefix)) continue;
      const uint32_t b = (o >> shift) & ((1u << bits) - 1);
      if (by_mass) {
        const u64 w = smp_weight(r, x);
        if (w == 0) continue;
        const unsigned lo = static_cast<unsigned>(w);
        const unsigned old = atomicAdd(&sh->mass[0][b], lo);
        const unsigned hi = static_cast<unsigned>(w >> 32) + (old + lo < old ? 1u : 0u);
        if (hi) atomicAdd(&sh->mass[1][b], hi);
      }
      atomicAdd(&sh->cnt[b], 1u);
    }
    cluster_sync();
    // thread t holds bins from the top: index i = t * kPer + q is bin last - i
    u64 c[kPer], v[kPer], sum = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int b = kSmpRadix - 1 - (tid * kPer + q);
      c[q] = v[q] = 0;
      for (int k = 0; k < r.ranks; ++k) {
        c[q] += ld_peer_u32(&sh->cnt[b], k);
        if (by_mass)
          v[q] += ld_peer_u32(&sh->mass[0][b], k) +
                  (static_cast<u64>(ld_peer_u32(&sh->mass[1][b], k)) << 32);
      }
      if (!by_mass) v[q] = c[q];
      sum += v[q];
    }
    u64 run = smp_block_scan(sh, sum);
    if (level == 0 && by_mass) {
      if (tid == kSmpThreads - 1) sh->bcast[0] = run;
      __syncthreads();
      goal = fmax(top_p * static_cast<double>(sh->bcast[0]), 1.0);   // the first is kept
    }
    run = base + run - sum;
    // the last bin that holds tokens and starts before the goal: the one in
    // which it is reached (or, if rounding lets none reach it, the last of all)
    if (tid == 0) sh->bcast[1] = 0;
    __syncthreads();
    int hit = -1;
    u64 hit_base = 0, hit_cnt = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (c[q] && (by_mass ? static_cast<double>(run) < goal : run < want)) {
        hit = kSmpRadix - 1 - (tid * kPer + q);
        hit_base = run;
        hit_cnt = c[q];
      }
      run += v[q];
    }
    if (hit >= 0)
      atomicMax(&sh->bcast[1], (static_cast<u64>(tid + 1) << 32) | static_cast<u64>(hit));
    __syncthreads();
    const u64 best = sh->bcast[1];
    if (static_cast<int>(best >> 32) == tid + 1) {
      sh->bcast[2] = hit_base;
      sh->bcast[3] = hit_cnt;
    }
    __syncthreads();
    prefix = (prefix << bits) | static_cast<uint32_t>(best);
    base = sh->bcast[2];
    bin_cnt = sh->bcast[3];
    cluster_sync();          // the histograms are cleared next
  }
  // all bin_cnt tokens here have the same value: how many of them are kept
  const float tau = smp_value(prefix);
  u64 n_keep;
  if (by_mass) {
    const u64 w = smp_weight(r, tau);
    const double over = (goal - static_cast<double>(base)) / static_cast<double>(w);
    n_keep = over >= static_cast<double>(bin_cnt) ? bin_cnt : static_cast<u64>(over);
    while (n_keep < bin_cnt && static_cast<double>(base + n_keep * w) < goal) ++n_keep;
    while (n_keep > 1 && static_cast<double>(base + (n_keep - 1) * w) >= goal) --n_keep;
  } else {
    n_keep = want - base;
  }
  if (n_keep < 1) n_keep = 1;
  if (n_keep > bin_cnt) n_keep = bin_cnt;
  // the n_keep-th tie in vocabulary order: warps own runs of the slice
  const int seg = ((r.len + kSmpWarps - 1) / kSmpWarps + 31) / 32 * 32;
  const int beg = min(r.len, warp * seg), end = min(r.len, beg + seg);
  const u64 tie_lo = max(floor_key, static_cast<u64>(prefix) << 32);
  const u64 tie_hi = (static_cast<u64>(prefix) << 32) | 0xffffffffull;
  u64 mine = 0;
  for (int i = beg + lane; i < end; i += 32) {
    const u64 key = smp_key(r.x[i], r.begin + i);
    mine += key >= tie_lo && key <= tie_hi;
  }
  const u64 in_warp = warp_sum_u64(mine);
  const u64 upto = smp_block_scan(sh, lane == 0 ? in_warp : 0ull);
  const u64 warp_end = __shfl_sync(0xffffffffu, upto, 0);
  if (tid == kSmpThreads - 1) sh->ties[which] = upto;
  if (tid == 0) sh->border[which] = 0;
  cluster_sync();
  u64 before = 0;
  for (int k = 0; k < r.rank; ++k) before += ld_peer_u64(&sh->ties[which], k);
  u64 at = before + warp_end - in_warp;
  if (at < n_keep && n_keep <= at + in_warp) {
    for (int i0 = beg; i0 < end; i0 += 32) {
      const int i = i0 + lane;
      const u64 key = i < end ? smp_key(r.x[i], r.begin + i) : 0ull;
      const bool tie = i < end && key >= tie_lo && key <= tie_hi;
      const unsigned b = __ballot_sync(0xffffffffu, tie);
      const u64 rank_here = at + __popc(b & ((1u << lane) - 1)) + 1;
      if (tie && rank_here == n_keep) sh->border[which] = key;
      at += __popc(b);
    }
  }
  cluster_sync();
  u64 key = 0;
  for (int k = 0; k < r.ranks; ++k) key = max(key, ld_peer_u64(&sh->border[which], k));
  return key;
}

struct SmpResult {
  int writer;      // this thread holds the result
  int accepted;    // the draft was taken
  int token;       // the drawn token, -1: nothing to draw from
  float prob;      // its share of the kept weight
};

__device__ __forceinline__ float smp_unit(float u) {   // into [0, 1)
  return u > 0.f ? fminf(u, 0.99999994f) : 0.f;
}

// Draw from the tokens with key >= floor_key in vocabulary order, over all of
// the row.  draft >= 0: first offered for acceptance with u_accept.
__device__ SmpResult smp_draw_row(const SmpRow& r, u64 floor_key, int draft, float u_accept,
                                  float u) {
  SmpShared* sh = r.sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = ((r.len + kSmpWarps - 1) / kSmpWarps + 31) / 32 * 32;
  const int beg = min(r.len, warp * seg), end = min(r.len, beg + seg);
  const int draft_at = draft - r.begin;
  u64 mine = 0, dw = 0;
  for (int i = beg + lane; i < end; i += 32) {
    const float x = r.x[i];
    if (smp_key(x, r.begin + i) < floor_key) continue;
    const u64 w = smp_weight(r, x);
    mine += w;
    if (i == draft_at) dw = w;
  }
  const u64 in_warp = warp_sum_u64(mine);
  dw = warp_sum_u64(dw);
  if (tid == 0) sh->draft_w = 0;
  const u64 upto = smp_block_scan(sh, lane == 0 ? in_warp : 0ull);
  if (lane == 0 && dw) sh->draft_w = dw;
  if (tid == kSmpThreads - 1) sh->kept = upto;
  cluster_sync();
  u64 before = 0, total = 0, draft_w = 0;
  int draft_rank = -1;
  for (int k = 0; k < r.ranks; ++k) {
    const u64 s = ld_peer_u64(&sh->kept, k);
    const u64 d = ld_peer_u64(&sh->draft_w, k);
    if (k < r.rank) before += s;
    total += s;
    draft_w += d;
    if (d) draft_rank = k;
  }
  cluster_sync();   // no CTA leaves while another reads its shared memory
  SmpResult out = {0, 0, -1, 0.f};
  if (draft >= 0 && draft_w > 0 &&
      (draft_w == total ||
       static_cast<double>(u_accept) * static_cast<double>(total) < static_cast<double>(draft_w))) {
    out.writer = r.rank == 0 && tid == 0;
    out.accepted = 1;
    out.token = draft;
    return out;
  }
  if (draft >= 0) {
    total -= draft_w;
    if (draft_rank >= 0 && draft_rank < r.rank) before -= draft_w;
  }
  if (total == 0) {
    out.writer = r.rank == 0 && tid == 0;
    return out;
  }
  const double goal = static_cast<double>(smp_unit(u)) * static_cast<double>(total);
  // the warp in whose run the running sum passes the goal
  const u64 warp_all = __shfl_sync(0xffffffffu, upto, 0);
  u64 end_sum = before + warp_all, run = end_sum - in_warp;
  if (draft >= 0 && draft_rank == r.rank) {
    if (draft_at < beg) run -= draft_w;
    if (draft_at < end) end_sum -= draft_w;
  }
  if (static_cast<double>(run) > goal || static_cast<double>(end_sum) <= goal || run == end_sum)
    return out;
  for (int i0 = beg; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    u64 w = 0;
    if (i < end && (draft < 0 || i != draft_at)) {
      const float x = r.x[i];
      if (smp_key(x, r.begin + i) >= floor_key) w = smp_weight(r, x);
    }
    const u64 upto_i = run + warp_scan_u64(w, lane);
    const unsigned b = __ballot_sync(0xffffffffu, static_cast<double>(upto_i) > goal);
    if (b) {
      if (lane == __ffs(b) - 1) {
        out.writer = 1;
        out.token = r.begin + i;
        out.prob = static_cast<float>(static_cast<double>(w) / static_cast<double>(total));
      }
      return out;
    }
    run = __shfl_sync(0xffffffffu, upto_i, 31);
  }
  return out;
}

// The same from n candidates in rank 0's list (keys in any order; every token
// that is kept is among them).  mass_all: the weight that top_p refers to, 0:
// that of the candidates.  Called by every thread of rank 0.
__device__ SmpResult smp_draw_list(const SmpRow& r, int n, int k, double top_p, u64 mass_all,
                                   int draft, float u_accept, float u) {
  SmpShared* sh = r.sh;
  const int tid = threadIdx.x;
  SmpResult out = {0, 0, -1, 0.f};
  int n2 = 32;
  while (n2 < n) n2 <<= 1;
  for (int i = n + tid; i < n2; i += kSmpThreads) sh->list[i] = 0;
  smp_sort(sh->list, n2);
  if (tid == 0) {
    sh->first_bad = n;
    sh->draft_w = 0;
  }
  // running weights in falling order: two neighbours a thread
  const int i0 = 2 * tid;
  u64 w[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = i0 + q;
    if (i < n && (k <= 0 || i < k))
      w[q] = smp_weight(r, smp_value(static_cast<uint32_t>(sh->list[i] >> 32)));
  }
  u64 run = smp_block_scan(sh, w[0] + w[1]);
  if (tid == kSmpThreads - 1) sh->bcast[0] = run;
  __syncthreads();
  run -= w[0] + w[1];
  const double goal =
      top_p * static_cast<double>(mass_all ? mass_all : sh->bcast[0]);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = i0 + q;
    if (i < n && i > 0 && (w[q] == 0 || !(static_cast<double>(run) < goal)))
      atomicMin(&sh->first_bad, static_cast<unsigned>(i));
    run += w[q];
    if (i < n) sh->w[i] = w[q];
  }
  __syncthreads();
  n = sh->first_bad;            // the kept tokens are list[0 .. n)
  n2 = 32;
  while (n2 < n) n2 <<= 1;
  // into vocabulary order, each with its place in w
  u64 key[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = i0 + q;
    key[q] = 0;
    if (i < n) {
      const uint32_t id = smp_id(sh->list[i]);
      key[q] = (static_cast<u64>(0xffffffffu - id) << 32) | static_cast<u64>(i);
      if (static_cast<int>(id) == draft) sh->draft_w = w[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (i0 + q < n2) sh->list[i0 + q] = key[q];
  smp_sort(sh->list, n2);
  const u64 draft_w = sh->draft_w;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = i0 + q;
    key[q] = i < n ? sh->list[i] : 0;
    w[q] = i < n ? sh->w[static_cast<uint32_t>(key[q])] : 0;
  }
  u64 total = smp_block_sum(sh, w[0] + w[1]);
  if (draft >= 0 && draft_w > 0 &&
      (draft_w == total ||
       static_cast<double>(u_accept) * static_cast<double>(total) < static_cast<double>(draft_w))) {
    out.writer = tid == 0;
    out.accepted = 1;
    out.token = draft;
    return out;
  }
  int id[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    id[q] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key[q] >> 32));
    if (i0 + q < n && id[q] == draft) w[q] = 0;
  }
  if (draft >= 0) total -= draft_w;
  if (total == 0) {
    out.writer = tid == 0;
    return out;
  }
  const double at = static_cast<double>(smp_unit(u)) * static_cast<double>(total);
  run = smp_block_scan(sh, w[0] + w[1]) - w[0] - w[1];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (!(static_cast<double>(run) > at) && static_cast<double>(run + w[q]) > at) {
      out.writer = 1;
      out.token = id[q];
      out.prob = static_cast<float>(static_cast<double>(w[q]) / static_cast<double>(total));
    }
    run += w[q];
  }
  return out;
}

// One row: copy, filters, draw.  Exactly one thread of the cluster returns with
// writer set.
__device__ SmpResult smp_row(SmpShared* sh, float* xs, const float* row, int V, int slice,
                             const SampleSettings& set, int at, int draft, float u_accept,
                             float u) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  SmpRow r;
  r.sh = sh;
  r.x = xs;
  r.rank = static_cast<int>(cluster_rank());
  r.ranks = gridDim.x;
  r.begin = r.rank * slice;
  r.len = max(0, min(V - r.begin, slice));
  const float* src = row + r.begin;
  if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
    for (int i = tid * 4; i + 4 <= r.len; i += kSmpThreads * 4) cp_async16(xs + i, src + i);
    for (int i = (r.len & ~3) + tid; i < r.len; i += kSmpThreads) cp_async4(xs + i, src + i);
  } else {
    for (int i = tid; i < r.len; i += kSmpThreads) cp_async4(xs + i, src + i);
  }
  const float T = set.temperature ? set.temperature[at] : 1.f;
  const int k_in = set.top_k ? set.top_k[at] : 0;
  const float p_in = set.top_p ? set.top_p[at] : 1.f;
  const float m_in = set.min_p ? set.min_p[at] : 0.f;
  if (tid < 32) sh->tab[tid] = exp2(tid / 32.0);
  for (int i = tid; i < kSmpBins; i += kSmpThreads) sh->cnt[i] = 0;
  cp_async_wait_all();
  __syncthreads();
  // largest (value, id) and smallest finite value
  float bv = -INFINITY, lo = INFINITY;
  int bi = -1;
  for (int i = tid; i < r.len; i += kSmpThreads) {
    float x = xs[i];
    x = x != x ? -INFINITY : x + 0.f;
    xs[i] = x;
    if (x > bv) {
      bv = x;
      bi = i;
    }
    if (x > -INFINITY) lo = fminf(lo, x);
  }
  u64 key = bi >= 0 ? smp_key(bv, r.begin + bi) : 0ull;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 other = __shfl_xor_sync(0xffffffffu, key, o);
    key = other > key ? other : key;
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  if (lane == 0) {
    sh->warp_a[warp] = key;
    reinterpret_cast<float*>(sh->mass)[warp] = lo;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kSmpWarps; ++w) {
      key = max(key, sh->warp_a[w]);
      lo = fminf(lo, reinterpret_cast<float*>(sh->mass)[w]);
    }
    sh->top_key = key;
    sh->low = lo;
  }
  cluster_sync();
  key = 0;
  lo = INFINITY;
  for (int k = 0; k < r.ranks; ++k) {
    key = max(key, ld_peer_u64(&sh->top_key, k));
    lo = fminf(lo, __uint_as_float(ld_peer_u32(&sh->low, k)));
  }
  SmpResult out = {r.rank == 0 && tid == 0, 0, -1, 0.f};
  if (key == 0) {              // nothing but -inf and NaN
    cluster_sync();
    return out;
  }
  r.m = smp_value(static_cast<uint32_t>(key >> 32));
  if (!(T > 0.f)) {            // greedy
    cluster_sync();
    out.token = static_cast<int>(smp_id(key));
    out.accepted = out.token == draft;
    out.prob = 1.f;
    return out;
  }
  r.c = 1.4426950408889634 / static_cast<double>(T);
  r.w_min = m_in > 0.f ? static_cast<u64>(ceil(fmin(m_in, 1.0) * 17592186044416.0)) : 0ull;
  const bool by_k = k_in > 0 && k_in < V;
  const bool by_p = p_in < 1.f;
  const double top_p = p_in > 0.f ? static_cast<double>(p_in) : 0.0;
  if (!by_k && !by_p) return smp_draw_row(r, 0ull, draft, u_accept, u);
  // How many tokens lie how far below the largest: linear bins of m - x down to
  // where a token weighs nothing.  s m - s x rounds monotonely, so each bin
  // holds a run of the falling order.
  const float reach = fminf(kSmpReach * T, r.m - lo);
  const float scale = (kSmpBins - 0.5f) / fmaxf(reach, 1e-30f);
  auto bin_of = [&](float x) {   // kSmpBins: too far down
    const float d = x == r.m ? 0.f : (r.m - x) * scale;
    return d < static_cast<float>(kSmpBins) ? static_cast<int>(d) : kSmpBins;
  };
  for (int i = tid; i < r.len; i += kSmpThreads) {
    const int b = bin_of(xs[i]);
    if (b < kSmpBins) atomicAdd(&sh->cnt[b], 1u);
  }
  // top_p without top_k: the weight it refers to is the whole row's
  u64 mass_all = 0;
  if (!by_k) {
    u64 mine = 0;
    for (int i = tid; i < r.len; i += kSmpThreads) mine += smp_weight(r, xs[i]);
    mine = smp_block_sum(sh, mine);
    if (tid == 0) sh->mass_all = mine;
  }
  cluster_sync();
  if (!by_k)
    for (int k = 0; k < r.ranks; ++k) mass_all += ld_peer_u64(&sh->mass_all, k);
  // the first bin by which every kept token has come: top_k tokens, or top_p
  // of the weight even if every token of a bin weighs as little as its far edge
  // (whose rounding, 46 bits times 2^-22, the factor 1.0001 covers)
  u64 c[2] = {0, 0}, earlier[2] = {0, 0};
  const double edge = -r.c / static_cast<double>(scale);
#pragma unroll
  for (int q = 0; q < 2; ++q)
    for (int k = 0; k < r.ranks; ++k) {
      const u64 v = ld_peer_u32(&sh->cnt[2 * tid + q], k);
      c[q] += v;
      if (k < r.rank) earlier[q] += v;
    }
  const u64 need = static_cast<u64>(by_k ? k_in : 0);
  u64 upto, measure[2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    measure[q] = by_k ? c[q]
                      : static_cast<u64>(static_cast<double>(c[q]) *
                                         exp2(edge * (2 * tid + q + 1.0) + kSmpOneBits));
  upto = smp_block_scan(sh, measure[0] + measure[1]);
  const u64 goal = by_k ? need
                        : static_cast<u64>(top_p * static_cast<double>(mass_all) * 1.0001) + 1;
  if (tid == 0) sh->first_bad = kSmpBins - 1;
  __syncthreads();
  if (upto >= goal) {
    const int b = upto - measure[1] >= goal ? 2 * tid : 2 * tid + 1;
    atomicMin(&sh->first_bad, static_cast<unsigned>(b));
  }
  __syncthreads();
  const int last_bin = static_cast<int>(sh->first_bad);
  u64 in = 0, off = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (2 * tid + q <= last_bin) {
      in += c[q];
      off += earlier[q];
    }
  in = smp_block_sum(sh, in);
  off = smp_block_sum(sh, off);
  if (in <= kSmpList) {
    if (tid == 0) sh->n_local = 0;
    __syncthreads();
    for (int i = tid; i < r.len; i += kSmpThreads) {
      const float x = xs[i];
      if (bin_of(x) <= last_bin) {
        const u64 at_i = off + atomicAdd(&sh->n_local, 1u);
        if (at_i < kSmpList) st_peer_u64(&sh->list[at_i], 0, smp_key(x, r.begin + i));
      }
    }
    cluster_sync();
    if (r.rank != 0) {
      out.writer = 0;
      return out;
    }
    return smp_draw_list(r, static_cast<int>(in), by_k ? k_in : 0, by_p ? top_p : 2.0, mass_all,
                         draft, u_accept, u);
  }
  // too many candidates for one list: exact borders over the whole row
  cluster_sync();
  u64 floor_key = 0;
  if (by_k) floor_key = smp_border(r, false, 0ull, need, 0.0, 0);
  if (by_p) floor_key = smp_border(r, true, floor_key, 0ull, top_p, 1);
  return smp_draw_row(r, floor_key, draft, u_accept, u);
}

struct SampleParams {
  const float* logits;
  int64_t ld;
  int rows, V, slice;
  SampleSettings set;
  const float* u;
  int32_t* tokens;
  float* probs;
  unsigned* err;
};

// Cluster y draws row y's token.
__global__ void __launch_bounds__(kSmpThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smp_smem[];
  pdl_trigger();
  pdl_wait();
  SmpShared* sh = reinterpret_cast<SmpShared*>(smp_smem);
  float* xs = reinterpret_cast<float*>(smp_smem + (sizeof(SmpShared) + 15) / 16 * 16);
  const int row = blockIdx.y;
  const SmpResult res = smp_row(sh, xs, p.logits + static_cast<int64_t>(row) * p.ld, p.V, p.slice,
                                p.set, row, -1, 0.f, p.u[row]);
  if (res.writer) {
    p.tokens[row] = res.token;
    if (p.probs) p.probs[row] = res.prob;
    if (res.token < 0) raise_error(p.err, DFLASH_DEVERR_INPUT);
  }
}

struct VerifySampledParams {
  const int32_t* drafts;
  const float* logits;
  int64_t ld;
  int B, K, V, slice;
  SampleSettings set;
  const float *u_accept, *u_sample;
  int32_t *out, *num_accepted, *bonus;
  unsigned* err;
  unsigned* done;         // [B] rows of the request that are settled (zeroed before)
  unsigned* refused;      // [B] K + 1 - (first refused row), 0: none yet (zeroed before)
  int32_t* row_token;     // [B][K + 1] what a row would emit if it is the last
};

// Cluster (y, z) settles row z of request y: rows come in order, so when a late
// row starts, an earlier one of its request may have refused its draft, and the
// row has nothing to say.  Whether it looks only decides if work is saved: a
// request's answer is its first refusing row's, whoever ran.  The cluster that
// settles a request's last row writes the answer.
__global__ void __launch_bounds__(kSmpThreads, 2)
verify_sampled_kernel(const VerifySampledParams p) {
  extern __shared__ __align__(16) uint8_t smp_smem[];
  pdl_trigger();
  pdl_wait();
  SmpShared* sh = reinterpret_cast<SmpShared*>(smp_smem);
  float* xs = reinterpret_cast<float*>(smp_smem + (sizeof(SmpShared) + 15) / 16 * 16);
  const int b = blockIdx.y, i = blockIdx.z, K = p.K;
  // one reading for the whole cluster: rank 0's
  if (threadIdx.x == 0 && cluster_rank() == 0)
    sh->n_local = *reinterpret_cast<volatile unsigned*>(p.refused + b);
  cluster_sync();
  const int refused = static_cast<int>(ld_peer_u32(&sh->n_local, 0));
  cluster_sync();
  SmpResult res = {0, 0, -1, 0.f};
  if (refused && i > K + 1 - refused) {
    res.writer = cluster_rank() == 0 && threadIdx.x == 0;
    res.accepted = 1;      // a row that does not matter
  } else {
    const int draft = i < K ? p.drafts[static_cast<int64_t>(b) * K + i] : -1;
    res = smp_row(sh, xs, p.logits + (static_cast<int64_t>(b) * (K + 1) + i) * p.ld, p.V, p.slice,
                  p.set, b, draft, i < K ? p.u_accept[static_cast<int64_t>(b) * K + i] : 0.f,
                  p.u_sample[b]);
  }
  if (!res.writer) return;
  if (!res.accepted || i == K) {
    p.row_token[static_cast<int64_t>(b) * (K + 1) + i] = res.token;
    __threadfence();
    atomicMax(p.refused + b, static_cast<unsigned>(K + 1 - i));
  }
  __threadfence();
  if (atomicAdd(p.done + b, 1u) != static_cast<unsigned>(K)) return;
  __threadfence();
  const int n = K + 1 - static_cast<int>(*reinterpret_cast<volatile unsigned*>(p.refused + b));
  const int32_t last =
      *reinterpret_cast<volatile int32_t*>(p.row_token + static_cast<int64_t>(b) * (K + 1) + n);
  int32_t* o = p.out + static_cast<int64_t>(b) * (K + 1);
  for (int j = 0; j <= K; ++j)
    o[j] = j < n ? p.drafts[static_cast<int64_t>(b) * K + j] : j == n ? last : -1;
  p.num_accepted[b] = n;
  p.bonus[b] = last;
  if (last < 0) raise_error(p.err, DFLASH_DEVERR_INPUT);
}

}  // namespace dflash
