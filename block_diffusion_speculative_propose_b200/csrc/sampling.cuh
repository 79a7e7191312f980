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
// Layout.  A cluster takes a row, each of its CTAs a slice.  The first pass
// brings the row from memory and finds the maxima; whatever the filters then
// need is read again while it still lies in L2, so a CTA holds no tokens and four
// of them share an SM, which hides what a row waits for (three cluster barriers
// and the tail in which one CTA sorts).  What the CTAs have to tell one another
// is pushed into each other's shared memory before a barrier.
//
// Work.  Only a row without top_k needs the weight of every token (the sums that
// u and top_p refer to); it costs about nine 64-bit operations.  A top_k needs
// no second pass: the k-th largest of the threads' own maxima bounds the k-th
// largest token from below, and only threads whose maximum reaches that bound
// look at their tokens again.  The candidates, a few more than k, are sorted.
#pragma once

#include "dflash_device.cuh"

namespace dflash {

constexpr int kSmpThreads = 256;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpCtas = 4;           // of an SM
constexpr int kSmpMaxCluster = 8;
constexpr int kSmpBins = 1024;        // linear bins of x below the maximum
constexpr int kSmpRadix = 2048;       // bins of a radix level (11 bits)
constexpr int kSmpList = 1024;        // candidates that one CTA sorts
constexpr int kSmpFew = 128;          // candidates that are ranked by comparing all pairs
constexpr int kSmpListTopK = 640;     // largest top_k whose candidates are gathered by maxima
constexpr int kSmpOneBits = 44;       // W of the largest weight: 2^44
constexpr float kSmpReach = 31.9f;    // 46 ln 2: tokens further below weigh nothing
constexpr int kSmpTab = 512;          // 2^(j / 512)
constexpr int kSmpMaxVocab = 393216;  // V 2^44 < 2^63

typedef unsigned long long u64;

struct SampleSettings {
  const float* temperature;   // one entry per row (or request); null: 1
  const int32_t* top_k;       // null or <= 0: off
  const float* top_p;         // null: 1
  const float* min_p;         // null: 0
};

// Every field that a peer writes or reads is used once a row, so a barrier
// between the writing and the reading is all it needs.
struct SmpShared {
  double tab[kSmpTab];
  u64 warp_a[kSmpWarps];             // block-wide sums
  u64 bcast[5];
  u64 kept_in[kSmpMaxCluster];       // from each rank: its kept weight, the draft's
  u64 draft_in[kSmpMaxCluster];
  u64 ties_in[2][kSmpMaxCluster];    // from each rank: ties of the border value (two searches)
  u64 border[2];                     // the border key (two searches)
  u64 told, n_keep;                  // from rank 0: how a search goes on
  float top_in[kSmpMaxCluster];      // from each rank: the largest value of its slice
  float thr_in[kSmpMaxCluster][4];   // and values that ever fewer of its tokens reach
  float thr[4];
  unsigned first_in[kSmpMaxCluster]; // greedy: the first id that holds the largest value
  unsigned first;
  unsigned n_list[4];                // rank 0: candidates gathered (four lists)
  unsigned n_own, own_at;            // this CTA's share of them, its place
  unsigned verdict, told32;          // from rank 0
  unsigned first_bad;
  union {
    __align__(16) unsigned cnt[kSmpRadix];   // histogram: tokens
    u64 own[kSmpList];                       // this CTA's candidates
  };
  union {
    __align__(16) unsigned mass[2][kSmpRadix];   // histogram: low, high words of weights
    struct {
      u64 list[kSmpList];                        // rank 0: the candidates' keys
      u64 w[kSmpList];
    };
  };
};

__device__ __forceinline__ float smp_norm(float x) {       // NaN as -inf, -0 as +0
  return fmaxf(x, -INFINITY) + 0.f;
}
__device__ __forceinline__ uint32_t smp_order(float x) {   // orders like x (no NaN, no -0)
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float smp_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ float smp_key_value(u64 key) {
  return smp_value(static_cast<uint32_t>(key >> 32));
}
__device__ __forceinline__ u64 smp_key(float x, uint32_t id) {
  return (static_cast<u64>(smp_order(x)) << 32) | (0xffffffffu - id);
}
__device__ __forceinline__ uint32_t smp_id(u64 key) {
  return 0xffffffffu - static_cast<uint32_t>(key);
}

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint4 ld_peer_v4(const void* p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(peer_addr(p, rank))
               : "memory");
  return v;
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
__device__ __forceinline__ void st_peer_u32(void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_peer_u32(void* p, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(peer_addr(p, rank)), "r"(v)
               : "memory");
  return old;
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

// The block's shared memory, in a form from which every function sees that it is shared.
__device__ __forceinline__ SmpShared* smp_shared() {
  extern __shared__ __align__(16) uint8_t smp_smem[];
  return reinterpret_cast<SmpShared*>(smp_smem);
}

// One row as the cluster's threads see it.
struct SmpRow {
  const float* x;        // this CTA's slice
  int len, padded, begin;   // its length, that rounded up to whole warp loads, its first id
  bool wide;             // its 16-byte loads are aligned
  int rank, ranks;
  float m;               // the row's largest value
  float x_cut;           // weighs nothing
  double md, c;          // m, 512 log2(e) / T
  u64 w_min;             // min_p as a weight
  bool fast;             // x_cut is between 46 and 60 bits below m
};

// Tokens i .. i+3 of the slice, -inf past its end (i a multiple of four).
__device__ __forceinline__ float4 smp_load4(const SmpRow& r, int i) {
  if (r.wide && i + 4 <= r.len) return __ldg(reinterpret_cast<const float4*>(r.x + i));
  float4 v;
  v.x = i < r.len ? __ldg(r.x + i) : -INFINITY;
  v.y = i + 1 < r.len ? __ldg(r.x + i + 1) : -INFINITY;
  v.z = i + 2 < r.len ? __ldg(r.x + i + 2) : -INFINITY;
  v.w = i + 3 < r.len ? __ldg(r.x + i + 3) : -INFINITY;
  return v;
}

// f(x, i) for tokens x[0..3] = i .. i+3 of the slice, all of it (-inf in its
// padding), four loads in flight a thread.  f works on four tokens at a time so
// that their chains of 64-bit operations overlap: at 40 cycles an operation and
// eight warps an SM's quarter they bound a pass otherwise.
template <class F>
__device__ __forceinline__ void smp_each(const SmpRow& r, F f) {
  for (int i0 = threadIdx.x * 4; i0 < r.padded; i0 += kSmpThreads * 16) {
    float4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q * kSmpThreads * 4;
      if (i < r.padded) v[q] = smp_load4(r, i);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q * kSmpThreads * 4;
      if (i >= r.padded) break;
      const float x[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
      f(x, i);
    }
  }
}

// An integer W plus kSmpBias, the bits of 2^52: sums of these wrap, and the
// bias is taken out of a sum at its end.
constexpr u64 kSmpBias = 0x4330000000000000ull;

// W + bias of value x: with t = (x - m) log2(e) / T = n/512 + f / 512,
// 2^t = 2^(n >> 9) 2^((n & 511) / 512) 2^(f / 512), |f| <= 1/2: three terms of
// the last factor's Taylor series leave (ln 2 / 1024)^4 / 24 < 2^-46.
__device__ __forceinline__ u64 smp_bits(const SmpRow& r, float x) {
  const double d = static_cast<double>(fmaxf(x, r.x_cut)) - r.md;   // a NaN is cut too
  const double magic = 6755399441055744.0;   // 1.5 2^52: the sum's low bits are the integer
  const double s = __fma_rn(d, r.c, magic);
  const int n = __double2loint(s);
  const double f = __fma_rn(d, r.c, magic - s);
  constexpr double a = 0.6931471805599453 / kSmpTab;   // ln 2 / 512
  double p = __fma_rn(f, a * a * a / 6.0, a * a / 2.0);
  p = __fma_rn(p, f, a);
  p = __fma_rn(p, f, 1.0);
  p *= smp_shared()->tab[n & (kSmpTab - 1)];
  // times 2^((n >> 9) + 44) (a normal number: n >> 9 >= -61), then the integer nearest
  const double v = __hiloint2double(__double2hiint(p) + (((n >> 9) + kSmpOneBits) << 20),
                                    __double2loint(p));
  return static_cast<u64>(__double_as_longlong(v + 4503599627370496.0));
}

// W of value x: 0 where it is filtered by min_p or weighs nothing.
__device__ __forceinline__ u64 smp_weight(const SmpRow& r, float x) {
  u64 w;
  if (r.fast) {
    w = smp_bits(r, x) - kSmpBias;
  } else if (x == r.m) {
    w = 1ull << kSmpOneBits;
  } else {
    // a temperature so small, or so large, or values so large that no cut in
    // fp32 serves: the same by the library's exponential
    const double t = (static_cast<double>(x) - r.md) * r.c / kSmpTab + kSmpOneBits;
    w = t >= -2.0 ? static_cast<u64>(__double2ll_rn(exp2(t))) : 0ull;   // NaN: 0
  }
  return w < r.w_min ? 0ull : w;
}

// Block-wide sum; every thread gets it.
__device__ __forceinline__ u64 smp_block_sum(u64 v) {
  SmpShared* sh = smp_shared();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum_u64(v);
  __syncthreads();
  if (lane == 0) sh->warp_a[warp] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kSmpWarps; ++w) v += sh->warp_a[w];
  return v;
}
// Block-wide inclusive scan of one value a thread (in thread order).
__device__ __forceinline__ u64 smp_block_scan(u64 v) {
  SmpShared* sh = smp_shared();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_scan_u64(v, lane);
  __syncthreads();
  if (lane == 31) sh->warp_a[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSmpWarps; ++w)
    if (w < warp) v += sh->warp_a[w];
  return v;
}

// Falling bitonic sort of list[0..n), n <= kSmpList.
__device__ __noinline__ void smp_sort(int n) {
  u64* a = smp_shared()->list;
  const int tid = threadIdx.x;
  int n2 = 64;
  while (n2 < n) n2 <<= 1;
  for (int i = n + tid; i < n2; i += kSmpThreads) a[i] = 0;
  for (int k = 2; k <= n2; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int i = tid; i < n2 / 2; i += kSmpThreads) {
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

// The linear bin of x below the maximum: fp32 2^23 + (m - x) scale rounds to an
// integer, and its bits order like it (a NaN comes last).
__device__ __forceinline__ unsigned smp_bin(float m, float scale, float x) {
  return __float_as_uint(fmaf(m - x, scale, 8388608.f)) - 0x4B000000u;
}

// One candidate into this CTA's own list / that list into rank 0's, counted in
// n_list[which] (past its room nothing is stored, only counted).
__device__ __forceinline__ void smp_candidate(float x, int id) {
  SmpShared* sh = smp_shared();
  const unsigned at = atomicAdd(&sh->n_own, 1u);
  if (at < kSmpList) sh->own[at] = smp_key(smp_norm(x), id);
}
__device__ __forceinline__ void smp_hand_over(int which) {
  SmpShared* sh = smp_shared();
  __syncthreads();
  const unsigned n = sh->n_own;
  if (threadIdx.x == 0 && n) sh->own_at = add_peer_u32(&sh->n_list[which], 0, n);
  __syncthreads();
  const unsigned at = sh->own_at;
  for (unsigned i = threadIdx.x; i < min(n, static_cast<unsigned>(kSmpList)) && at + i < kSmpList;
       i += kSmpThreads)
    st_peer_u64(&sh->list[at + i], 0, sh->own[i]);
}

__device__ __forceinline__ void smp_clear(int bins, bool by_mass) {
  SmpShared* sh = smp_shared();
  for (int i = threadIdx.x; i < bins; i += kSmpThreads) {
    sh->cnt[i] = 0;
    if (by_mass) {
      sh->mass[0][i] = 0;
      sh->mass[1][i] = 0;
    }
  }
  __syncthreads();
}
__device__ __forceinline__ void smp_count(unsigned b, bool by_mass, u64 w) {
  SmpShared* sh = smp_shared();
  if (by_mass) {
    const unsigned lo = static_cast<unsigned>(w);
    const unsigned old = atomicAdd(&sh->mass[0][b], lo);
    const unsigned hi = static_cast<unsigned>(w >> 32) + (old + lo < old ? 1u : 0u);
    if (hi) atomicAdd(&sh->mass[1][b], hi);
  }
  atomicAdd(&sh->cnt[b], 1u);
}

// Sums over the ranks of four neighbouring bins, all loads in flight at once:
// f32(e, sum) and f64(e, sum) get bin e's, which fits either.
template <class F32, class F64>
__device__ __forceinline__ void smp_bins_of_all(const unsigned* bins, int ranks, F32 f32,
                                                F64 f64) {
  uint4 n[kSmpMaxCluster];
#pragma unroll
  for (int k = 0; k < kSmpMaxCluster; ++k)
    n[k] = k < ranks ? ld_peer_v4(bins, k) : make_uint4(0, 0, 0, 0);
  u64 t[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < kSmpMaxCluster; ++k) {
    t[0] += n[k].x;
    t[1] += n[k].y;
    t[2] += n[k].z;
    t[3] += n[k].w;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f32(e, static_cast<unsigned>(t[e]));
    f64(e, t[e]);
  }
}

struct SmpHit {
  unsigned bin;      // in the histogram
  u64 base, cnt;     // the measure before it, its tokens
  u64 all;           // the measure of all bins
  u64 upto;          // tokens before and in it
};
// Rank 0: the last bin that holds anything and starts before the goal - the one in
// which it is reached, or, if rounding lets none reach it, the last of all.
// Bins are taken in rising order, or (falling) from the last one down.  With
// top_p >= 0 the goal becomes top_p of all.
template <int BINS>
__device__ SmpHit smp_merge(const SmpRow& r, bool by_mass, bool falling, u64 base, double top_p,
                            double& goal) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  constexpr int kPer = BINS / kSmpThreads;   // bins of a thread, a multiple of four
  u64 v[kPer];
  unsigned c[kPer];
#pragma unroll
  for (int q = 0; q < kPer; q += 4) {
    const int b = (falling ? BINS - kPer - tid * kPer : tid * kPer) + q;
    smp_bins_of_all(&sh->cnt[b], r.ranks, [&](int e, unsigned n) {
      c[q + e] = n;
    }, [&](int e, u64 n) { v[q + e] = n; });
    if (by_mass) {
      smp_bins_of_all(&sh->mass[0][b], r.ranks, [&](int, unsigned) {},
                      [&](int e, u64 n) { v[q + e] = n; });
      smp_bins_of_all(&sh->mass[1][b], r.ranks, [&](int, unsigned) {},
                      [&](int e, u64 n) { v[q + e] += n << 32; });
    }
  }
  u64 sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) sum += v[q];
  u64 run = smp_block_scan(sum);
  u64 tokens = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) tokens += c[q];
  tokens = smp_block_scan(tokens) - tokens;
  if (tid == kSmpThreads - 1) sh->bcast[0] = run;
  if (tid == 0) sh->bcast[1] = 0;
  __syncthreads();
  SmpHit h;
  h.all = sh->bcast[0];
  if (top_p >= 0.0) goal = fmax(top_p * static_cast<double>(h.all), 1.0);   // the first is kept
  run += base - sum;
  int hit = -1;
  u64 hit_base = 0, hit_cnt = 0, hit_upto = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int q = falling ? kPer - 1 - j : j;
    tokens += c[q];
    if (c[q] && static_cast<double>(run) < goal) {
      hit = (falling ? BINS - kPer - tid * kPer : tid * kPer) + q;
      hit_base = run;
      hit_cnt = c[q];
      hit_upto = tokens;
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
    sh->bcast[4] = hit_upto;
  }
  __syncthreads();
  h.bin = static_cast<unsigned>(best);
  h.base = sh->bcast[2];
  h.cnt = sh->bcast[3];
  h.upto = sh->bcast[4];
  return h;
}
// Rank 0 tells every CTA; read as sh->told behind the next cluster barrier.
__device__ __forceinline__ void smp_tell(const SmpRow& r, u64 v) {
  if (threadIdx.x < r.ranks) st_peer_u64(&smp_shared()->told, threadIdx.x, v);
}

// The border of a kept prefix among the tokens with key >= floor_key: the key
// of the `want`-th of them (by_mass false), or of the first at which their
// running weight reaches top_p of all of theirs.  Every CTA of the cluster
// takes part and gets the same answer.  `which` (0, 1) separates the shared
// fields of a row's two searches.
//
// Three radix levels find the value, then the ties at it are counted in
// vocabulary order: right for any values, slow where many share a bin.
__device__ __noinline__ u64 smp_border_radix(const SmpRow r, bool by_mass, u64 floor_key,
                                             u64 want, double top_p, int which) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t prefix = 0;
  u64 base = 0;             // rank 0: tokens, or weight, above the current prefix
  u64 ties = 0;             // rank 0: tokens of the final value
  double goal = static_cast<double>(want);
  for (int level = 0; level < 3; ++level) {
    const int bits = level == 2 ? 10 : 11;
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
    smp_clear(kSmpRadix, by_mass);
    smp_each(r, [&](const float (&raw)[4], int i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = smp_norm(raw[q]);
        const u64 key = smp_key(x, r.begin + i + q);
        const uint32_t o = static_cast<uint32_t>(key >> 32);
        if (i + q >= r.len || key < floor_key || (level > 0 && (o >> (shift + bits)) != prefix))
          continue;
        u64 w = 0;
        if (by_mass && (w = smp_weight(r, x)) == 0) continue;
        smp_count((o >> shift) & ((1u << bits) - 1), by_mass, w);
      }
    });
    cluster_sync();
    if (r.rank == 0) {
      const SmpHit h = smp_merge<kSmpRadix>(r, by_mass, true, base,
                                            by_mass && level == 0 ? top_p : -1.0, goal);
      base = h.base;
      ties = h.cnt;
      smp_tell(r, h.bin);
    }
    cluster_sync();
    prefix = (prefix << bits) | static_cast<uint32_t>(sh->told);
  }
  // all tokens of this value weigh the same: how many of them are kept
  if (r.rank == 0) {
    u64 n_keep;
    if (by_mass) {
      const u64 w = smp_weight(r, smp_value(prefix));
      const double over = (goal - static_cast<double>(base)) / static_cast<double>(w);
      n_keep = over >= static_cast<double>(ties) ? ties : static_cast<u64>(over);
      while (n_keep < ties && static_cast<double>(base + n_keep * w) < goal) ++n_keep;
      while (n_keep > 1 && static_cast<double>(base + (n_keep - 1) * w) >= goal) --n_keep;
    } else {
      n_keep = want - base;
    }
    n_keep = max(1ull, min(ties, n_keep));
    if (tid < r.ranks) st_peer_u64(&sh->n_keep, tid, n_keep);
  }
  // the n_keep-th tie in vocabulary order: warps own runs of the slice
  const int seg = ((r.len + kSmpWarps - 1) / kSmpWarps + 31) / 32 * 32;
  const int beg = min(r.len, warp * seg), end = min(r.len, beg + seg);
  const u64 tie_lo = max(floor_key, static_cast<u64>(prefix) << 32);
  const u64 tie_hi = (static_cast<u64>(prefix) << 32) | 0xffffffffull;
  u64 mine = 0;
  for (int i = beg + lane; i < end; i += 32) {
    const u64 key = smp_key(smp_norm(__ldg(r.x + i)), r.begin + i);
    mine += key >= tie_lo && key <= tie_hi;
  }
  const u64 in_warp = warp_sum_u64(mine);
  const u64 upto = smp_block_scan(lane == 0 ? in_warp : 0ull);
  const u64 warp_end = __shfl_sync(0xffffffffu, upto, 0);
  if (tid == kSmpThreads - 1)
    for (int k = 0; k < r.ranks; ++k) st_peer_u64(&sh->ties_in[which][r.rank], k, upto);
  cluster_sync();
  const u64 n_keep = sh->n_keep;
  u64 at = warp_end - in_warp;
  for (int k = 0; k < r.rank; ++k) at += sh->ties_in[which][k];
  if (at < n_keep && n_keep <= at + in_warp) {
    for (int i0 = beg; i0 < end; i0 += 32) {
      const int i = i0 + lane;
      const u64 key = i < end ? smp_key(smp_norm(__ldg(r.x + i)), r.begin + i) : 0ull;
      const bool tie = i < end && key >= tie_lo && key <= tie_hi;
      const unsigned b = __ballot_sync(0xffffffffu, tie);
      const u64 rank_here = at + __popc(b & ((1u << lane) - 1)) + 1;
      if (tie && rank_here == n_keep)
        for (int k = 0; k < r.ranks; ++k) st_peer_u64(&sh->border[which], k, key);
      at += __popc(b);
    }
  }
  cluster_sync();
  return sh->border[which];
}

// Tokens of one bin of a histogram into rank 0's list, and of them the border:
// the first at which `base` and their running measure reach the goal (base and
// goal are rank 0's).
template <class BinAt>
__device__ __forceinline__ u64 smp_border_in_bin(const SmpRow& r, BinAt bin_at, unsigned bin,
                                                 bool by_mass, u64 base, double goal, int which) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  smp_each(r, [&](const float (&x)[4], int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (bin_at(x[q], i + q) == bin) smp_candidate(x[q], r.begin + i + q);
  });
  smp_hand_over(1 + which);
  cluster_sync();
  if (r.rank == 0) {
    const int n = min(sh->n_list[1 + which], static_cast<unsigned>(kSmpList));
    smp_sort(n);
    constexpr int kPer = kSmpList / kSmpThreads;
    const int i0 = kPer * tid;
    u64 w[kPer], sum = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      w[q] = i0 + q < n ? (by_mass ? smp_weight(r, smp_key_value(sh->list[i0 + q])) : 1ull) : 0ull;
      sum += w[q];
    }
    u64 at = base + smp_block_scan(sum) - sum;
    if (tid == 0) sh->first_bad = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (w[q] && static_cast<double>(at) < goal) atomicMax(&sh->first_bad, i0 + q);
      at += w[q];
    }
    __syncthreads();
    if (tid < r.ranks) st_peer_u64(&sh->border[which], tid, sh->list[sh->first_bad]);
  }
  cluster_sync();
  return sh->border[which];
}

// What rank 0 tells besides a bin.
constexpr u64 kSmpRefine = 1ull << 32, kSmpNothing = 2ull << 32;

// The border of top_k = want: a histogram of linear bins below the maximum, of
// the bin in which the border lies if that holds more than a list, and the
// sorted list.  The radix search where even that holds more (ties).
__device__ __noinline__ u64 smp_border_k(const SmpRow r, float scale, u64 want) {
  SmpShared* sh = smp_shared();
  if (!r.fast) return smp_border_radix(r, false, 0ull, want, 0.0, 0);
  unsigned bin = 0;
  float shift = 0.f;         // second level: (m - x) scale - shift spans [0, 1]
  u64 base = 0;              // rank 0
  double goal = static_cast<double>(want);
  int level = 0;
  // kSmpBins or more: not looked at
  auto bin_at = [&](float x, int) -> unsigned {
    const unsigned b = smp_bin(r.m, scale, x);
    if (level == 0) return b;
    if (b != bin) return kSmpBins;
    const float f = fmaxf(fmaf(r.m - x, scale, -shift), 0.f);
    return min(__float_as_uint(fmaf(f, kSmpBins - 2.f, 8388608.f)) - 0x4B000000u, kSmpBins - 1u);
  };
  for (;; ++level) {
    smp_clear(kSmpBins, false);
    smp_each(r, [&](const float (&x)[4], int i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned b = bin_at(x[q], i + q);
        if (b < kSmpBins) atomicAdd(&sh->cnt[b], 1u);
      }
    });
    cluster_sync();
    if (r.rank == 0) {
      const SmpHit h = smp_merge<kSmpBins>(r, false, false, base, -1.0, goal);
      base = h.base;
      // fewer than wanted weigh anything: nothing to cut
      smp_tell(r, level == 0 && h.all < want ? kSmpNothing
                  : h.cnt > kSmpList         ? kSmpRefine | h.bin
                                             : h.bin);
    }
    if (threadIdx.x == 0) sh->n_own = 0;
    cluster_sync();
    const u64 told = sh->told;
    if (told >= kSmpNothing) return 0ull;
    if (told < kSmpRefine)
      return smp_border_in_bin(r, bin_at, static_cast<unsigned>(told), false, base, goal, 0);
    if (level) return smp_border_radix(r, false, 0ull, want, 0.0, 0);
    bin = static_cast<unsigned>(told);
    shift = static_cast<float>(bin) - 0.5f;
  }
}

// top_p over the tokens with key >= floor_key: a histogram of their weights in
// linear bins, of the bin in which the border lies if that holds more than a
// list, and the sorted list.  Sums of integers are exact, so the bins say exactly
// where the border lies.  If a list can hold all tokens up to it, the list is
// filled (`listed` is set, rank 0 has the weight of all in mass_all) and the
// caller draws from it.  The radix search where even the second histogram leaves
// too many (ties).
__device__ __noinline__ u64 smp_border_p(const SmpRow r, float scale, u64 floor_key,
                                         double top_p, bool* listed, u64* mass_all) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  *listed = false;
  if (!r.fast) return smp_border_radix(r, true, floor_key, 0ull, top_p, 1);
  const float tau = floor_key ? smp_key_value(floor_key) : -INFINITY;
  const int last = floor_key ? static_cast<int>(smp_id(floor_key)) - r.begin : 0x7fffffff;
  const bool plain = floor_key == 0 && r.w_min == 0;
  auto kept = [&](float x, int i) { return x > tau || (x == tau && i <= last); };
  scale *= static_cast<float>(kSmpRadix / kSmpBins);    // finer bins: a weight costs more
  unsigned bin = 0;
  float shift = 0.f;         // second level: (m - x) scale - shift spans [0, 1]
  int level = 0;
  // kSmpRadix or more: not looked at
  auto bin_at = [&](float x, int i) -> unsigned {
    const unsigned b = smp_bin(r.m, scale, x);
    if (!plain && !kept(x, i)) return kSmpRadix;
    if (level == 0) return b;
    if (b != bin) return kSmpRadix;
    const float f = fmaxf(fmaf(r.m - x, scale, -shift), 0.f);
    return min(__float_as_uint(fmaf(f, kSmpRadix - 2.f, 8388608.f)) - 0x4B000000u,
               kSmpRadix - 1u);
  };
  u64 base = 0;              // rank 0
  double goal = 0.0;
  for (;; ++level) {
    smp_clear(kSmpRadix, true);
    smp_each(r, [&](const float (&x)[4], int i) {
      unsigned b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) b[q] = bin_at(x[q], i + q);
      if (min(min(b[0], b[1]), min(b[2], b[3])) >= kSmpRadix) return;
      u64 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = smp_bits(r, x[q]) - kSmpBias;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (b[q] < kSmpRadix && w[q] && w[q] >= r.w_min) smp_count(b[q], true, w[q]);
    });
    cluster_sync();
    if (r.rank == 0) {
      const SmpHit h = smp_merge<kSmpRadix>(r, true, false, base, level == 0 ? top_p : -1.0, goal);
      base = h.base;
      if (level == 0) *mass_all = h.all;
      smp_tell(r, level == 0 && h.upto <= kSmpList ? kSmpNothing | h.bin
                  : h.cnt > kSmpList               ? kSmpRefine | h.bin
                                                   : h.bin);
    }
    if (tid == 0) sh->n_own = 0;
    cluster_sync();
    const u64 told = sh->told;
    bin = level == 0 ? static_cast<unsigned>(told) : bin;
    if (told >= kSmpNothing) break;
    if (told < kSmpRefine)
      return smp_border_in_bin(r, bin_at, static_cast<unsigned>(told), true, base, goal, 1);
    if (level) return smp_border_radix(r, true, floor_key, 0ull, top_p, 1);
    shift = static_cast<float>(bin) - 0.5f;
  }
  smp_each(r, [&](const float (&x)[4], int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (bin_at(x[q], i + q) <= bin) smp_candidate(x[q], r.begin + i + q);
  });
  smp_hand_over(3);
  cluster_sync();
  // tokens of these bins that min_p filters are in the list too
  *listed = ld_peer_u32(&sh->n_list[3], 0) <= kSmpList;
  cluster_sync();
  return *listed ? floor_key : smp_border_radix(r, true, floor_key, 0ull, top_p, 1);
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
__device__ __forceinline__ bool smp_accepts(u64 draft_w, u64 total, float u_accept) {
  return draft_w > 0 && (draft_w == total || static_cast<double>(u_accept) *
                                                     static_cast<double>(total) <
                                                 static_cast<double>(draft_w));
}
__device__ __forceinline__ float smp_share(u64 w, u64 total) {
  return static_cast<float>(static_cast<double>(w) / static_cast<double>(total));
}

// Draw from the tokens with key >= floor_key in vocabulary order, over all of
// the row.  draft >= 0: first offered for acceptance with u_accept.
__device__ __forceinline__ SmpResult smp_draw_row(const SmpRow& r, u64 floor_key, int draft,
                                                  float u_accept, float u) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float tau = floor_key ? smp_key_value(floor_key) : -INFINITY;
  const int last = floor_key ? static_cast<int>(smp_id(floor_key)) - r.begin : 0x7fffffff;
  // kept: above the border's value, or at it and not behind its id
  auto keep = [&](float x, int i) { return x > tau || (x == tau && i <= last); };
  auto weight = [&](float x, int i) -> u64 { return keep(x, i) ? smp_weight(r, x) : 0ull; };
  // warps own runs of 128-token groups, a lane four neighbours of a group
  const int seg = ((r.padded >> 7) + kSmpWarps - 1) / kSmpWarps * 128;
  const int beg = min(r.padded, warp * seg), end = min(r.padded, beg + seg);
  const int draft_at = draft - r.begin;
  u64 mine = 0;
  if (r.fast && r.w_min == 0) {
    for (int i0 = beg + lane * 4; i0 < end; i0 += 512) {
      float4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i0 + q * 128 < end) v[q] = smp_load4(r, i0 + q * 128);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + q * 128;
        if (i >= end) break;
        const u64 a = smp_bits(r, v[q].x), b = smp_bits(r, v[q].y), c = smp_bits(r, v[q].z),
                  d = smp_bits(r, v[q].w);
        if (floor_key == 0) {
          mine += a + b;
          mine += c + d;
          mine -= 4 * kSmpBias;
        } else {
          mine += (keep(v[q].x, i) ? a - kSmpBias : 0) + (keep(v[q].y, i + 1) ? b - kSmpBias : 0);
          mine += (keep(v[q].z, i + 2) ? c - kSmpBias : 0) +
                  (keep(v[q].w, i + 3) ? d - kSmpBias : 0);
        }
      }
    }
  } else {
    for (int i = beg + lane * 4; i < end; i += 128) {
      const float4 v = smp_load4(r, i);
      mine += weight(v.x, i) + weight(v.y, i + 1) + weight(v.z, i + 2) + weight(v.w, i + 3);
    }
  }
  const u64 in_warp = warp_sum_u64(mine);
  const u64 upto = smp_block_scan(lane == 0 ? in_warp : 0ull);
  if (tid == kSmpThreads - 1) {
    const u64 d = draft >= 0 && draft_at >= 0 && draft_at < r.len
                      ? weight(__ldg(r.x + draft_at), draft_at)
                      : 0ull;
    for (int k = 0; k < r.ranks; ++k) {
      st_peer_u64(&sh->kept_in[r.rank], k, upto);
      st_peer_u64(&sh->draft_in[r.rank], k, d);
    }
  }
  if (tid == 0) sh->first_bad = kSmpWarps;
  cluster_sync();   // the row's last: no CTA touches another's memory behind it
  u64 before = 0, total = 0, draft_w = 0;
  int draft_rank = -1;
  for (int k = 0; k < r.ranks; ++k) {
    const u64 s = sh->kept_in[k], d = sh->draft_in[k];
    if (k < r.rank) before += s;
    total += s;
    draft_w += d;
    if (d) draft_rank = k;
  }
  SmpResult out = {0, 0, -1, 0.f};
  if (smp_accepts(draft_w, total, u_accept)) {
    out.writer = r.rank == 0 && tid == 0;
    out.accepted = 1;
    out.token = draft;
    return out;
  }
  total -= draft_w;
  if (draft_rank >= 0 && draft_rank < r.rank) before -= draft_w;
  if (total == 0) {
    out.writer = r.rank == 0 && tid == 0;
    return out;
  }
  const double goal = static_cast<double>(smp_unit(u)) * static_cast<double>(total);
  // the warp in whose run the running sum passes the goal
  const u64 warp_all = __shfl_sync(0xffffffffu, upto, 0);
  u64 end_sum = before + warp_all, run = end_sum - in_warp;
  if (draft_rank == r.rank) {
    if (draft_at < beg) run -= draft_w;
    if (draft_at < end) end_sum -= draft_w;
  }
  if (lane == 0 && run != end_sum && !(static_cast<double>(run) > goal) &&
      static_cast<double>(end_sum) > goal) {
    sh->first_bad = warp;
    sh->bcast[0] = run;
  }
  __syncthreads();
  if (sh->first_bad >= kSmpWarps) return out;    // not in this slice
  // the CTA scans that run together, eight neighbours a thread
  const int b0 = static_cast<int>(sh->first_bad) * seg, b1 = min(r.padded, b0 + seg);
  run = sh->bcast[0];
  for (int i0 = b0; i0 < b1; i0 += kSmpThreads * 4) {
    const int i = i0 + tid * 4;
    float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (i < b1) {
      const float4 v = smp_load4(r, i);
      x[0] = v.x;
      x[1] = v.y;
      x[2] = v.z;
      x[3] = v.w;
    }
    u64 w[4], sum = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = i >= b1 || (draft_w && draft_rank == r.rank && i + q == draft_at)
                 ? 0ull
                 : weight(x[q], i + q);
      sum += w[q];
    }
    u64 at = run + smp_block_scan(sum);
    if (tid == kSmpThreads - 1) sh->bcast[1] = at;
    at -= sum;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (w[q] && !(static_cast<double>(at) > goal) && static_cast<double>(at + w[q]) > goal) {
        out.writer = 1;
        out.token = r.begin + i + q;
        out.prob = smp_share(w[q], total);
      }
      at += w[q];
    }
    __syncthreads();
    run = sh->bcast[1];
  }
  return out;
}

// The same from n candidates in rank 0's list (keys in any order; every token
// that is kept is among them).  mass_all: the weight that top_p refers to, 0:
// that of the first k candidates.  Called by every thread of rank 0.
__device__ __forceinline__ SmpResult smp_draw_few(const SmpRow& r, int n, int k, double top_p,
                                                  u64 mass_all, int draft, float u_accept,
                                                  float u) {
  // n <= kSmpFew: kShare threads compare a candidate with all others, so its
  // place, and the weight before it in either order, need no sort
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  constexpr int kShare = kSmpThreads / kSmpFew;
  const int i = tid / kShare, q0 = tid % kShare;
  SmpResult out = {0, 0, -1, 0.f};
  if (tid < n) sh->w[tid] = smp_weight(r, smp_key_value(sh->list[tid]));
  __syncthreads();
  const u64 key = i < n ? sh->list[i] : 0ull;
  u64 w = i < n ? sh->w[i] : 0ull, before = 0;
  int place = 0;
  for (int j = q0; j < n; j += kShare)
    if (sh->list[j] > key) {
      ++place;
      before += sh->w[j];
    }
#pragma unroll
  for (int o = 1; o < kShare; o <<= 1) {
    place += __shfl_xor_sync(0xffffffffu, place, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (k <= 0 || k > n) k = n;
  if (i < n && q0 == 0 && place == k - 1) sh->bcast[0] = before + w;
  __syncthreads();
  const double goal = top_p * static_cast<double>(mass_all ? mass_all : sh->bcast[0]);
  if (place >= k || (place > 0 && !(static_cast<double>(before) < goal))) w = 0;
  if (i < n && q0 == 0) sh->w[i] = w;
  __syncthreads();
  const uint32_t id = smp_id(key);
  u64 total = 0, draft_w = 0;
  before = 0;
  for (int j = q0; j < n; j += kShare) {
    const u64 wj = sh->w[j];
    const uint32_t idj = smp_id(sh->list[j]);
    total += wj;
    if (static_cast<int>(idj) == draft) draft_w += wj;
    else if (idj < id) before += wj;
  }
#pragma unroll
  for (int o = 1; o < kShare; o <<= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    draft_w += __shfl_xor_sync(0xffffffffu, draft_w, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (smp_accepts(draft_w, total, u_accept)) {
    out.writer = tid == 0;
    out.accepted = 1;
    out.token = draft;
    return out;
  }
  total -= draft_w;
  if (total == 0) {
    out.writer = tid == 0;
    return out;
  }
  const double at = static_cast<double>(smp_unit(u)) * static_cast<double>(total);
  if (i < n && q0 == 0 && w && static_cast<int>(id) != draft &&
      !(static_cast<double>(before) > at) && static_cast<double>(before + w) > at) {
    out.writer = 1;
    out.token = static_cast<int>(id);
    out.prob = smp_share(w, total);
  }
  return out;
}
__device__ __noinline__ SmpResult smp_draw_list(const SmpRow r, int n, int k, double top_p,
                                                u64 mass_all, int draft, float u_accept, float u) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  constexpr int kPer = kSmpList / kSmpThreads;
  SmpResult out = {0, 0, -1, 0.f};
  smp_sort(n);
  if (tid == 0) {
    sh->first_bad = n;
    sh->bcast[2] = 0;
  }
  // running weights in falling order: neighbours a thread
  const int i0 = kPer * tid;
  u64 w[kPer], sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = i0 + q;
    w[q] = i < n && (k <= 0 || i < k) ? smp_weight(r, smp_key_value(sh->list[i])) : 0ull;
    sum += w[q];
  }
  u64 run = smp_block_scan(sum);
  if (tid == kSmpThreads - 1) sh->bcast[0] = run;
  __syncthreads();
  run -= sum;
  const double goal = top_p * static_cast<double>(mass_all ? mass_all : sh->bcast[0]);
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = i0 + q;
    if (i < n && i > 0 && (w[q] == 0 || !(static_cast<double>(run) < goal)))
      atomicMin(&sh->first_bad, static_cast<unsigned>(i));
    run += w[q];
  }
  __syncthreads();
  n = sh->first_bad;            // the kept tokens are list[0 .. n)
  // into vocabulary order
  u64 key[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = i0 + q;
    key[q] = 0;
    if (i < n) {
      const u64 old = sh->list[i];
      if (static_cast<int>(smp_id(old)) == draft) sh->bcast[2] = w[q];
      key[q] = (old << 32) | (old >> 32);     // falling ~id first
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (i0 + q < n) sh->list[i0 + q] = key[q];
  smp_sort(n);
  const u64 draft_w = sh->bcast[2];
  int id[kPer];
  sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = i0 + q;
    key[q] = i < n ? sh->list[i] : 0;
    id[q] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key[q] >> 32));
    w[q] = i < n ? smp_weight(r, smp_value(static_cast<uint32_t>(key[q]))) : 0;
    if (id[q] == draft) w[q] = 0;
    sum += w[q];
  }
  run = smp_block_scan(sum);
  if (tid == kSmpThreads - 1) sh->bcast[1] = run;
  __syncthreads();
  const u64 total = sh->bcast[1];             // without the draft
  if (smp_accepts(draft_w, total + draft_w, u_accept)) {
    out.writer = tid == 0;
    out.accepted = 1;
    out.token = draft;
    return out;
  }
  if (total == 0) {
    out.writer = tid == 0;
    return out;
  }
  run -= sum;
  const double at = static_cast<double>(smp_unit(u)) * static_cast<double>(total);
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (w[q] && !(static_cast<double>(run) > at) && static_cast<double>(run + w[q]) > at) {
      out.writer = 1;
      out.token = id[q];
      out.prob = smp_share(w[q], total);
    }
    run += w[q];
  }
  return out;
}

// One row: maxima, filters, draw.  Exactly one thread of the cluster returns with
// writer set.
__device__ __forceinline__ SmpResult smp_row(const float* row, int V, int slice,
                                             const SampleSettings& set, int at, int draft,
                                             float u_accept, float u) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  SmpRow r;
  r.rank = static_cast<int>(cluster_rank());
  r.ranks = gridDim.x;
  r.begin = r.rank * slice;
  r.len = max(0, min(V - r.begin, slice));
  r.padded = (r.len + 127) & ~127;
  r.x = row + r.begin;
  r.wide = (reinterpret_cast<uintptr_t>(r.x) & 15) == 0;
  const float T = set.temperature ? set.temperature[at] : 1.f;
  const int k_in = set.top_k ? set.top_k[at] : 0;
  const float p_in = set.top_p ? set.top_p[at] : 1.f;
  const float m_in = set.min_p ? set.min_p[at] : 0.f;
  // the largest of this thread's tokens (a NaN never is); eight loads in flight
  float mine = -INFINITY;
  for (int i0 = tid * 4; i0 < r.padded; i0 += kSmpThreads * 32) {
    float4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int i = i0 + q * kSmpThreads * 4;
      v[q] = i < r.padded ? smp_load4(r, i)
                          : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      mine = fmaxf(mine, fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w)));
  }
  const bool greedy = !(T > 0.f);
  const bool by_k = k_in > 0 && k_in < V;
  const bool by_p = p_in < 1.f;
  const double top_p = p_in > 0.f ? static_cast<double>(p_in) : 0.0;
  const float scale = fminf((kSmpBins - 1) / (kSmpReach * T), 3e38f);
  const bool by_list = !greedy && by_k && k_in <= kSmpListTopK;
  if (!greedy) {
    for (int i = tid; i < kSmpTab; i += kSmpThreads) sh->tab[i] = exp2(i * (1.0 / kSmpTab));
    if (by_list)
      for (int i = tid; i < kSmpBins; i += kSmpThreads) sh->cnt[i] = 0;
  }
  if (tid < 4) sh->n_list[tid] = 0;
  if (tid < 4) sh->thr[tid] = -INFINITY;
  if (tid == 0) {
    sh->n_own = 0;
    sh->first = 0xffffffffu;
  }
  float top = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float* warp_f = reinterpret_cast<float*>(sh->warp_a);
  if (lane == 0) warp_f[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSmpWarps; ++w) top = fmaxf(top, warp_f[w]);
  if (by_list) {
    // thr[j]: a value that at least aim / 2^j of the slice's tokens reach, seen
    // from the threads' maxima alone (-inf where too few are within reach)
    const unsigned b = smp_bin(top, scale, mine);
    if (b < kSmpBins) atomicAdd(&sh->cnt[b], 1u);
    __syncthreads();
    constexpr int kPer = kSmpBins / kSmpThreads;
    unsigned c[kPer], sum = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      c[q] = sh->cnt[tid * kPer + q];
      sum += c[q];
    }
    unsigned run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned w = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += w;
    }
    unsigned* warp_u = reinterpret_cast<unsigned*>(sh->bcast);
    if (lane == 31) warp_u[warp] = run;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSmpWarps; ++w)
      if (w < warp) run += warp_u[w];
    run -= sum;
    const unsigned aim = static_cast<unsigned>(k_in);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned need = (aim + (1u << j) - 1) >> j;
        // below every value of that bin, whatever its rounding
        if (run < need && run + c[q] >= need)
          sh->thr[j] = __double2float_rd(static_cast<double>(top) -
                                         (tid * kPer + q + 0.51) / static_cast<double>(scale));
      }
      run += c[q];
    }
    __syncthreads();
  }
  if (tid < r.ranks) {
    st_peer_u32(&sh->top_in[r.rank], tid, __float_as_uint(top));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_peer_u32(&sh->thr_in[r.rank][j], tid, __float_as_uint(sh->thr[j]));
  }
  cluster_sync();
  // 2^j slices that hold aim / 2^j tokens each from a value on hold aim: the
  // 2^j-th largest of thr[j]; of the four such values the largest
  float cut = -INFINITY;
  {
    const int c = lane >> 2, j = lane & 3;
    top = lane < r.ranks ? sh->top_in[lane] : -INFINITY;
    if (by_list) {
      const float v = c < r.ranks ? sh->thr_in[c][j] : -INFINITY;
      int above = 0;
#pragma unroll
      for (int o = 1; o < 8; ++o) {
        const int from = ((c + o) & 7) * 4 + j;
        const float w = __shfl_sync(0xffffffffu, v, from);
        above += w > v || (w == v && from < lane);
      }
      cut = above == (1 << j) - 1 ? v : -INFINITY;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      cut = fmaxf(cut, __shfl_xor_sync(0xffffffffu, cut, o));
    }
  }
  r.m = top + 0.f;
  SmpResult out = {r.rank == 0 && tid == 0, 0, -1, 0.f};
  if (top == -INFINITY) return out;   // nothing but -inf and NaN
  if (greedy) {                       // the first id of the largest value
    if (mine == top)
      for (int i = tid * 4; i < r.padded; i += kSmpThreads * 4) {
        const float4 v = smp_load4(r, i);
        const int q = v.x == top ? 0 : v.y == top ? 1 : v.z == top ? 2 : v.w == top ? 3 : -1;
        if (q >= 0) {
          atomicMin(&sh->first, static_cast<unsigned>(r.begin + i + q));
          break;
        }
      }
    __syncthreads();
    if (tid == 0) st_peer_u32(&sh->first_in[r.rank], 0, sh->first);
    cluster_sync();
    unsigned id = 0xffffffffu;
    for (int k = 0; k < r.ranks; ++k) id = min(id, sh->first_in[k]);
    out.token = static_cast<int>(id);
    out.accepted = out.token == draft;
    out.prob = 1.f;
    return out;
  }
  r.md = static_cast<double>(r.m);
  r.c = kSmpTab * 1.4426950408889634 / static_cast<double>(T);
  r.w_min = m_in > 0.f ? static_cast<u64>(ceil(fmin(m_in, 1.0) * 17592186044416.0)) : 0ull;
  r.x_cut = __double2float_rd(r.md - 46.5 * kSmpTab / r.c);
  const double below = (r.md - static_cast<double>(r.x_cut)) * r.c;
  r.fast = r.x_cut > -INFINITY && r.m < INFINITY && below >= 46.0 * kSmpTab &&
           below <= 60.0 * kSmpTab;
  u64 floor_key = 0, mass_all = 0;
  bool listed = false;
  if (by_list && r.fast) {
    cut = fmaxf(cut, r.x_cut);         // tokens further down weigh nothing
    // a warp looks at the tokens of each of its threads that reached the cut
    for (unsigned hot = __ballot_sync(0xffffffffu, mine >= cut); hot; hot &= hot - 1) {
      const int of = (warp * 32 + __ffs(hot) - 1) * 4;
      for (int i = of + lane * kSmpThreads * 4; i < r.padded; i += kSmpThreads * 128) {
        const float4 v = smp_load4(r, i);
        if (v.x >= cut) smp_candidate(v.x, r.begin + i);
        if (v.y >= cut) smp_candidate(v.y, r.begin + i + 1);
        if (v.z >= cut) smp_candidate(v.z, r.begin + i + 2);
        if (v.w >= cut) smp_candidate(v.w, r.begin + i + 3);
      }
    }
    smp_hand_over(0);
    cluster_sync();
    if (r.rank == 0 && tid < r.ranks) st_peer_u32(&sh->verdict, tid, sh->n_list[0] <= kSmpList);
    cluster_sync();
    listed = sh->verdict != 0;
  }
  if (!listed) {
    if (by_k) floor_key = smp_border_k(r, scale, static_cast<u64>(k_in));
    if (by_p) floor_key = smp_border_p(r, scale, floor_key, top_p, &listed, &mass_all);
  }
  if (!listed) return smp_draw_row(r, floor_key, draft, u_accept, u);
  out.writer = 0;
  if (r.rank != 0) return out;
  const bool by_border = mass_all != 0;      // listed by border_p: top_k is done
  const int n = sh->n_list[by_border ? 3 : 0], k = by_k && !by_border ? k_in : 0;
  const double p = by_p ? top_p : 2.0;
  return n <= kSmpFew ? smp_draw_few(r, n, k, p, mass_all, draft, u_accept, u)
                      : smp_draw_list(r, n, k, p, mass_all, draft, u_accept, u);
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
__global__ void __launch_bounds__(kSmpThreads, kSmpCtas) sample_kernel(const SampleParams p) {
  pdl_trigger();
  pdl_wait();
  SmpShared* sh = smp_shared();
  const int row = blockIdx.y;
  const SmpResult res = smp_row(p.logits + static_cast<int64_t>(row) * p.ld, p.V, p.slice,
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
  int run;                // rows that one cluster settles in turn
};

// Cluster (y, z) settles rows [z * run, ..) of request y in turn, until one
// refuses its draft.  Clusters start in the order of z: when a late one starts,
// an earlier row of its request may have refused, and its rows have nothing to
// say.  Whether it looks only decides if work is saved: a request's answer is
// its first refusing row's, whoever ran.  The cluster that settles a request's
// last rows writes the answer.
__global__ void __launch_bounds__(kSmpThreads, kSmpCtas)
verify_sampled_kernel(const VerifySampledParams p) {
  pdl_trigger();
  pdl_wait();
  SmpShared* sh = smp_shared();
  const int b = blockIdx.y, K = p.K;
  const int first = blockIdx.z * p.run, end = min(K + 1, first + p.run);
  const bool lead = threadIdx.x == 0 && cluster_rank() == 0;
  bool needed = true;
  if (first > 0) {
    // one reading for the whole cluster: rank 0's
    if (lead) {
      const unsigned refused = *reinterpret_cast<volatile unsigned*>(p.refused + b);
      const unsigned told = !(refused && first > K + 1 - static_cast<int>(refused));
      for (unsigned k = 0; k < gridDim.x; ++k) st_peer_u32(&sh->verdict, k, told);
    }
    cluster_sync();
    needed = sh->verdict != 0;
    __syncthreads();
  }
  for (int i = first; needed && i < end; ++i) {
    const int draft = i < K ? p.drafts[static_cast<int64_t>(b) * K + i] : -1;
    const SmpResult res =
        smp_row(p.logits + (static_cast<int64_t>(b) * (K + 1) + i) * p.ld, p.V, p.slice, p.set,
                b, draft, i < K ? p.u_accept[static_cast<int64_t>(b) * K + i] : 0.f,
                p.u_sample[b]);
    if (res.writer && (!res.accepted || i == K)) {
      p.row_token[static_cast<int64_t>(b) * (K + 1) + i] = res.token;
      __threadfence();
      atomicMax(p.refused + b, static_cast<unsigned>(K + 1 - i));
      __threadfence();
    }
    // whether to go on (an accepted draft's writer is the leader); behind the
    // barrier the row's stores are out, for the leader to count it as settled
    if (lead) {
      const unsigned more = res.writer && res.accepted && i < K;
      for (unsigned k = 0; k < gridDim.x; ++k) st_peer_u32(&sh->told32, k, more);
    }
    cluster_sync();
    needed = sh->told32 != 0;
    cluster_sync();      // read by all before anything is written again
  }
  if (!lead) return;
  __threadfence();
  const unsigned mine = static_cast<unsigned>(end - first);
  if (atomicAdd(p.done + b, mine) + mine != static_cast<unsigned>(K + 1)) return;
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
