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
// of them share an SM, which hides what a row waits for (the cluster barriers and
// the tail in which one CTA works on a list).  What the CTAs have to tell one
// another is pushed into each other's shared memory before a barrier.
//
// Work.  Only a row without top_k needs the weight of every token (the sums that
// u and top_p refer to); it costs about nine 64-bit operations.  A top_k needs
// no second pass: the k-th largest of the threads' own maxima bounds the k-th
// largest token from below, and only threads whose maximum reaches that bound
// look at their tokens again.  The candidates, a few more than k, are ranked in
// one CTA.
//
// Measured (rows of 151936 unless said otherwise), against reading the rows once:
//   1 row, top_k 20, top_p 0.8       13 us: the chain of barriers and of 64-bit steps
//   16 rows of a verify              21 us: the same, and the clearing launch
//   512 rows of 128256, no filter   142 us: 41; the weights' 64-bit operations
//   320 rows of 128256, top_p 0.9   142 us: 25; two passes over weights, and the
//                                   histogram's shared-memory additions
//   128 rows, mixed filters          80 us: 12; the rows with top_p alone
//   128 requests of 16 rows, mixed  200 us: 192; rows behind a refusal are spared
// A wave is 74 rows (4 CTAs an SM, 8 a row); top_k rows take 20 us of it, rows
// that need all weights 40 to 75.
#pragma once

#include "dflash_device.cuh"

namespace dflash {

constexpr int kSmpThreads = 256;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpCtas = 4;           // of an SM
// CTAs of a row (the largest portable cluster).  Four suit a batch of top_k rows
// better (128 rows take 0.73 of the time), but a batch whose filters differ waits
// for its slowest rows (128 rows 1.33 of it), and of a request's rows fewer are
// spared (128 requests of 16 rows 1.36 of it).
constexpr int kSmpRanks = 8;
constexpr int kSmpBins = kSmpRanks * kSmpThreads;   // of a histogram: each thread merges one
constexpr int kSmpMaxBins = 1024;     // bins of the threads' maxima
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
  double tab[kSmpTab];               // 2^(44 + j / 512)
  u64 warp_a[kSmpWarps];             // block-wide sums
  u64 bcast[4];
  u64 all_in[2][kSmpRanks];          // from each rank: measure and tokens of its bins
  u64 hit[4];                        // from the rank that has it: bin, base, tokens, tokens up to it
  u64 kept_in[kSmpRanks];            // from each rank: its kept weight, the draft's
  u64 draft_in[kSmpRanks];
  u64 ties_in[2][kSmpRanks];         // from each rank: ties of the border value (two searches)
  u64 border[2];                     // the border key (two searches)
  float top_in[kSmpRanks];           // from each rank: the largest value of its slice
  float thr_in[kSmpRanks][4];        // and values that ever fewer of its tokens reach
  float thr[4];
  unsigned first_in[kSmpRanks];      // greedy: the first id that holds the largest value
  unsigned first;
  unsigned n_list[4];                // rank 0: candidates gathered (four lists)
  unsigned n_own, own_at;            // this CTA's share of them, its place
  unsigned verdict, more;            // from rank 0
  unsigned found, n_bucket;
  unsigned run_w[2][kSmpWarps];      // kept border tokens' weights by warp, low and high words
  union {
    unsigned cnt[kSmpBins];          // histogram: tokens
    u64 own[kSmpList];               // this CTA's candidates
    u64 bucket[kSmpList];            // rank 0: places in the list
  };
  union {
    unsigned mass[2][kSmpBins];      // histogram: low, high words of weights
    struct {
      u64 list[kSmpList];            // rank 0: the candidates' keys
      u64 w[kSmpList];               // and their weights
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

// The two halves of a cluster barrier that orders nothing.  Before a CTA touches a
// peer's memory the peer must have started: every CTA arrives before it reads the
// row, and waits when it has something to push, which costs nothing by then.
__device__ __forceinline__ void smp_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void smp_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
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
  int rank;
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
  // times 2^(n >> 9) (a normal number: n >> 9 >= -61), then the integer nearest
  const double v = __hiloint2double(__double2hiint(p) + (n & ~(kSmpTab - 1)) * (1 << 11),
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

__device__ __forceinline__ void smp_clear(bool tokens, bool weights) {
  SmpShared* sh = smp_shared();
  for (int i = threadIdx.x; i < kSmpBins; i += kSmpThreads) {
    if (tokens) sh->cnt[i] = 0;
    if (weights) {
      sh->mass[0][i] = 0;
      sh->mass[1][i] = 0;
    }
  }
  __syncthreads();
}
// 64-bit adds to shared memory would be a loop; two of 32 bits and a carry are not.
__device__ __forceinline__ void smp_add(unsigned* lo, unsigned* hi, u64 w) {
  const unsigned l = static_cast<unsigned>(w);
  const unsigned old = atomicAdd(lo, l);
  atomicAdd(hi, static_cast<unsigned>(w >> 32) + (old + l < old ? 1u : 0u));
}

// Which tokens a histogram's weights stand for, at most: bin b's weigh 2^-(t0 + (b +
// 0.51) dt) of the largest or more before they are rounded to integers, so a W is
// that less a half, and no less than 1.  dt 0: they are counted.
struct SmpDepth {
  double t0, dt;
};

struct SmpHit {
  unsigned bin;      // in the histogram
  u64 base, cnt;     // the measure before it, its tokens (counted, or at most)
  u64 all;           // the measure of all bins
  u64 upto;          // tokens before and in it
};
// The cluster's histograms together: the bin in which `base` and the running
// measure (weights, or tokens) reach the goal, or, if they never do, the last
// that holds anything.  Bins are taken in rising order, or (falling) from the
// last one down.  With top_p >= 0 the goal becomes top_p of all.  Each thread
// merges one bin over the CTAs; begins and ends with a cluster barrier, behind
// which every CTA has the answer.
__device__ __noinline__ SmpHit smp_find(int rank, bool by_mass, bool falling, u64 base,
                                        double top_p, SmpDepth depth, double* goal_io) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  const bool counted = depth.dt == 0.0;
  cluster_sync();
  const int at = rank * kSmpThreads + tid;
  const int b = falling ? kSmpBins - 1 - at : at;
  unsigned n[3][kSmpRanks];
#pragma unroll
  for (int k = 0; k < kSmpRanks; ++k) {
    n[0][k] = counted ? ld_peer_u32(&sh->cnt[b], k) : 0u;
    n[1][k] = by_mass ? ld_peer_u32(&sh->mass[0][b], k) : 0u;
    n[2][k] = by_mass ? ld_peer_u32(&sh->mass[1][b], k) : 0u;
  }
  u64 c = 0, v = 0;
#pragma unroll
  for (int k = 0; k < kSmpRanks; ++k) {
    c += n[0][k];
    v += n[1][k] + (static_cast<u64>(n[2][k]) << 32);
  }
  if (!by_mass) v = c;
  if (!counted && v) {
    const double least = exp2(kSmpOneBits - depth.t0 - (b + 0.51) * depth.dt) - 0.5;
    c = static_cast<u64>(static_cast<double>(v) / fmax(least, 1.0)) + 1;
  }
  const u64 run_v = smp_block_scan(v), run_c = smp_block_scan(c);
  if (tid == kSmpThreads - 1)
    for (int k = 0; k < kSmpRanks; ++k) {
      st_peer_u64(&sh->all_in[0][rank], k, run_v);
      st_peer_u64(&sh->all_in[1][rank], k, run_c);
    }
  cluster_sync();
  SmpHit h;
  u64 first = run_v - v, upto = run_c;
  h.all = 0;
#pragma unroll
  for (int k = 0; k < kSmpRanks; ++k) {
    if (k < rank) {
      first += sh->all_in[0][k];
      upto += sh->all_in[1][k];
    }
    h.all += sh->all_in[0][k];
  }
  double goal = *goal_io;
  if (top_p >= 0.0) *goal_io = goal = fmax(top_p * static_cast<double>(h.all), 1.0);   // keep one
  if (v && static_cast<double>(base + first) < goal &&
      (static_cast<double>(base + first + v) >= goal || first + v == h.all)) {
    for (int k = 0; k < kSmpRanks; ++k) {
      st_peer_u64(&sh->hit[0], k, b);
      st_peer_u64(&sh->hit[1], k, base + first);
      st_peer_u64(&sh->hit[2], k, c);
      st_peer_u64(&sh->hit[3], k, upto);
    }
  }
  cluster_sync();
  h.bin = static_cast<unsigned>(sh->hit[0]);
  h.base = sh->hit[1];
  h.cnt = sh->hit[2];
  h.upto = sh->hit[3];
  return h;
}

// Rank 0, all threads: among n listed tokens in the order of falling keys (by_id
// false) or rising ids, the one at which `base` and the running weights w[] reach
// the goal (pass: exceed it): its place in the list, -1 if none does; *before gets
// the sum in front of it.  A histogram of 256 buckets over the order leaves a
// few tokens that are compared with one another.
__device__ __noinline__ int smp_cross(int n, bool by_id, bool pass, u64 base, double goal,
                                      u64* before) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // falling keys are rising complements, whose low words are the ids
  auto order = [&](int i) -> u64 {
    const u64 key = ~sh->list[i];
    return by_id ? key & 0xffffffffull : key;
  };
  auto over = [&](u64 sum) {
    return pass ? static_cast<double>(sum) > goal : static_cast<double>(sum) >= goal;
  };
  u64 lo = ~0ull, hi = 0;
  for (int i = tid; i < n; i += kSmpThreads) {
    const u64 o = order(i);
    lo = min(lo, o);
    hi = max(hi, o);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  __syncthreads();
  if (lane == 0) {
    sh->warp_a[warp] = lo;
    reinterpret_cast<u64*>(sh->cnt)[warp] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSmpWarps; ++w) {
    lo = min(lo, sh->warp_a[w]);
    hi = max(hi, reinterpret_cast<u64*>(sh->cnt)[w]);
  }
  __syncthreads();
  unsigned* sum_lo = sh->cnt + 2 * kSmpList - 2 * kSmpThreads;   // behind the bucket's room
  unsigned* sum_hi = sum_lo + kSmpThreads;
  sum_lo[tid] = 0;
  sum_hi[tid] = 0;
  if (tid == 0) {
    sh->found = 0xffffffffu;
    sh->n_bucket = 0;
  }
  __syncthreads();
  const float per = (kSmpThreads - 0.5f) / (__ull2float_ru(hi - lo) + 1.f);
  auto bucket = [&](int i) {
    return min(static_cast<int>(__ull2float_rn(order(i) - lo) * per), kSmpThreads - 1);
  };
  for (int i = tid; i < n; i += kSmpThreads) {
    const int b = bucket(i);
    smp_add(&sum_lo[b], &sum_hi[b], sh->w[i]);
  }
  __syncthreads();
  const u64 v = sum_lo[tid] + (static_cast<u64>(sum_hi[tid]) << 32);
  const u64 run = base + smp_block_scan(v);
  if (v && over(run) && !over(run - v)) {
    sh->found = tid;
    sh->bcast[0] = run - v;
  }
  __syncthreads();
  const unsigned in = sh->found;
  if (in == 0xffffffffu) return -1;
  base = sh->bcast[0];
  __syncthreads();
  // the bucket's tokens: few, unless many keys lie together
  constexpr int kRoom = kSmpList - kSmpThreads;
  for (int i = tid; i < n; i += kSmpThreads)
    if (bucket(i) == static_cast<int>(in)) {
      const unsigned at = atomicAdd(&sh->n_bucket, 1u);
      if (at < kRoom) sh->bucket[at] = i;
    }
  if (tid == 0) sh->found = 0xffffffffu;
  __syncthreads();
  const unsigned nb = sh->n_bucket;
  const bool listed = nb <= kRoom;
  const int m = listed ? static_cast<int>(nb) : n;
  for (int a = tid; a < m; a += kSmpThreads) {
    const int i = listed ? static_cast<int>(sh->bucket[a]) : a;
    if (bucket(i) != static_cast<int>(in) || sh->w[i] == 0) continue;
    const u64 o = order(i);
    u64 sum = base;
    for (int c = 0; c < m; ++c) {
      const int j = listed ? static_cast<int>(sh->bucket[c]) : c;
      if ((listed || bucket(j) == static_cast<int>(in)) && order(j) < o) sum += sh->w[j];
    }
    if (over(sum + sh->w[i]) && !over(sum)) {
      sh->found = i;
      sh->bcast[0] = sum;
    }
  }
  __syncthreads();
  *before = sh->bcast[0];
  return static_cast<int>(sh->found);
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
  u64 base = 0;             // tokens, or weight, above the current prefix
  u64 ties = 0;             // tokens of the final value
  double goal = static_cast<double>(want);
  for (int level = 0; level < 3; ++level) {
    const int bits = level == 2 ? 10 : 11;
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
    smp_clear(true, by_mass);
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
        const uint32_t b = (o >> shift) & ((1u << bits) - 1);
        if (by_mass) smp_add(&sh->mass[0][b], &sh->mass[1][b], w);
        atomicAdd(&sh->cnt[b], 1u);
      }
    });
    const SmpHit h = smp_find(r.rank, by_mass, true, base, by_mass && level == 0 ? top_p : -1.0,
                              SmpDepth{0.0, 0.0}, &goal);
    base = h.base;
    ties = h.cnt;
    prefix = (prefix << bits) | h.bin;
  }
  // all tokens of this value weigh the same: how many of them are kept
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
    for (int k = 0; k < kSmpRanks; ++k) st_peer_u64(&sh->ties_in[which][r.rank], k, upto);
  cluster_sync();
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
        for (int k = 0; k < kSmpRanks; ++k) st_peer_u64(&sh->border[which], k, key);
      at += __popc(b);
    }
  }
  cluster_sync();
  return sh->border[which];
}

// Bins of a search's two levels: of m - x below the maximum, then the parts of
// the bin in which the border lies.
struct SmpBinning {
  float m, scale, shift;
  unsigned bin;
  int level;
  __device__ __forceinline__ unsigned sub(float x) const {
    const float f = fmaxf(fmaf(m - x, scale, -shift), 0.f);   // 0 .. 1
    return min(__float_as_uint(fmaf(f, kSmpBins - 2.f, 8388608.f)) - 0x4B000000u, kSmpBins - 1u);
  }
  // kSmpBins or more: not looked at
  __device__ __forceinline__ unsigned operator()(float x) const {
    const unsigned b = smp_bin(m, scale, x);
    if (level == 0) return b;
    return b == bin ? sub(x) : kSmpBins;
  }
  // before (negative), in (0) or behind bin `at` of the search's last level
  __device__ __forceinline__ int side(float x, unsigned at) const {
    const unsigned b = smp_bin(m, scale, x);
    if (level && b == bin) {
      const unsigned s = sub(x);
      return s < at ? -1 : s > at;
    }
    const unsigned t = level ? bin : at;
    return b < t ? -1 : b > t;
  }
  __device__ __forceinline__ void refine(unsigned b) {
    bin = b;
    shift = static_cast<float>(b) - 0.5f;
    level = 1;
  }
};

// Where a kept prefix ends: at a key, or (open) still somewhere in a bin, at the
// token at which `base` and the running measure of the bin's tokens with key >=
// floor reach the goal.
struct SmpBorder {
  u64 key;
  bool open, by_mass;
  SmpBinning bins;
  unsigned bin;
  u64 base, floor;
  double goal;
};
__device__ __forceinline__ SmpBorder smp_at_key(u64 key) {
  SmpBorder b;
  b.key = key;
  b.open = false;
  return b;
}

// The border's key, once the bin's tokens are in rank 0's list n_list[1 + which]: the
// search counted them, or bounded their number, so they all have room.
__device__ __forceinline__ u64 smp_close(const SmpRow& r, const SmpBorder& bd, int which) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  smp_hand_over(1 + which);
  cluster_sync();
  if (r.rank == 0) {
    const int n = min(sh->n_list[1 + which], static_cast<unsigned>(kSmpList));
    for (int i = tid; i < n; i += kSmpThreads)
      sh->w[i] = bd.by_mass ? smp_weight(r, smp_key_value(sh->list[i])) : 1ull;
    __syncthreads();
    u64 before;
    const int at = smp_cross(n, false, false, bd.base, bd.goal, &before);
    if (tid < kSmpRanks) st_peer_u64(&sh->border[which], tid, at >= 0 ? sh->list[at] : 0ull);
  }
  cluster_sync();
  return sh->border[which];
}
__device__ __forceinline__ u64 smp_resolve(const SmpRow& r, const SmpBorder& bd, int which) {
  if (!bd.open) return bd.key;
  if (threadIdx.x == 0) smp_shared()->n_own = 0;
  __syncthreads();
  smp_each(r, [&](const float (&x)[4], int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (bd.bins.side(x[q], bd.bin) == 0) smp_candidate(x[q], r.begin + i + q);
  });
  return smp_close(r, bd, which);
}

// The border of top_k = want: a histogram of linear bins below the maximum, and of
// the bin in which the border lies if that holds more than a list.  The radix
// search where even that holds more (ties).
__device__ __noinline__ SmpBorder smp_border_k(const SmpRow r, float scale, u64 want) {
  SmpShared* sh = smp_shared();
  if (!r.fast) return smp_at_key(smp_border_radix(r, false, 0ull, want, 0.0, 0));
  SmpBorder bd = {0, true, false, {r.m, scale, 0.f, 0u, 0}, 0, 0, 0, static_cast<double>(want)};
  for (;;) {
    smp_clear(true, false);
    smp_each(r, [&](const float (&x)[4], int) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned b = bd.bins(x[q]);
        if (b < kSmpBins) atomicAdd(&sh->cnt[b], 1u);
      }
    });
    const SmpHit h = smp_find(r.rank, false, false, bd.base, -1.0, SmpDepth{0.0, 0.0}, &bd.goal);
    if (bd.bins.level == 0 && h.all < want) return smp_at_key(0ull);   // fewer weigh anything
    bd.base = h.base;
    bd.bin = h.bin;
    if (h.cnt <= kSmpList) return bd;
    if (bd.bins.level) return smp_at_key(smp_border_radix(r, false, 0ull, want, 0.0, 0));
    bd.bins.refine(h.bin);
  }
}

// top_p over the tokens with key >= floor_key: the same with their weights.  Sums
// of integers are exact, so the bins say exactly where the border lies.  If a
// list can hold all tokens up to it, the list is filled and the caller draws
// from it (`listed`; mass_all is the weight of all that top_p refers to).
__device__ __noinline__ SmpBorder smp_border_p(const SmpRow r, float scale, u64 floor_key,
                                               double top_p, bool* listed, u64* mass_all) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x;
  *listed = false;
  if (!r.fast) return smp_at_key(smp_border_radix(r, true, floor_key, 0ull, top_p, 1));
  const float tau = floor_key ? smp_key_value(floor_key) : -INFINITY;
  const int last = floor_key ? static_cast<int>(smp_id(floor_key)) - r.begin : 0x7fffffff;
  SmpBorder bd = {0, true, true, {r.m, scale, 0.f, 0u, 0}, 0, 0, floor_key, 0.0};
  auto bin_at = [&](float x, int i) -> unsigned {
    const unsigned b = bd.bins(x);
    return floor_key == 0 || x > tau || (x == tau && i <= last) ? b : kSmpBins;
  };
  const double per_bin = r.c / kSmpTab / static_cast<double>(scale);
  SmpDepth depth = {0.0, per_bin};
  SmpHit h;
  for (;;) {
    smp_clear(false, true);
    smp_each(r, [&](const float (&x)[4], int i) {
      unsigned b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) b[q] = bin_at(x[q], i + q);
      if (min(min(b[0], b[1]), min(b[2], b[3])) >= kSmpBins) return;
      u64 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = smp_bits(r, x[q]) - kSmpBias;
      if (r.w_min) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (w[q] < r.w_min) b[q] = kSmpBins;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (b[q] < kSmpBins) smp_add(&sh->mass[0][b[q]], &sh->mass[1][b[q]], w[q]);
    });
    h = smp_find(r.rank, true, false, bd.base, bd.bins.level == 0 ? top_p : -1.0, depth, &bd.goal);
    bd.base = h.base;
    bd.bin = h.bin;
    if (bd.bins.level == 0) {
      *mass_all = h.all;
      if (h.upto <= kSmpList) break;
    }
    if (h.cnt <= kSmpList) return bd;
    if (bd.bins.level) return smp_at_key(smp_border_radix(r, true, floor_key, 0ull, top_p, 1));
    bd.bins.refine(h.bin);
    depth = {(h.bin - 0.5) * per_bin, per_bin / (kSmpBins - 2)};
  }
  if (tid == 0) sh->n_own = 0;
  __syncthreads();
  smp_each(r, [&](const float (&x)[4], int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (bin_at(x[q], i + q) <= h.bin) smp_candidate(x[q], r.begin + i + q);
  });
  smp_hand_over(3);
  cluster_sync();
  // more than counted only if min_p filters some of these bins' tokens
  if (r.rank == 0 && tid < kSmpRanks) st_peer_u32(&sh->verdict, tid, sh->n_list[3] <= kSmpList);
  cluster_sync();
  *listed = sh->verdict != 0;
  return smp_at_key(*listed ? floor_key
                            : smp_border_radix(r, true, floor_key, 0ull, top_p, 1));
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

// Draw from the tokens up to the border (all of them unless BORDER) in vocabulary
// order, over all of the row.  draft >= 0: first offered for acceptance with
// u_accept.
template <bool BORDER>
__device__ __forceinline__ SmpResult smp_draw_row(const SmpRow& r, const SmpBorder& bd, int draft,
                                                  float u_accept, float u) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // warps own runs of 128-token groups, a lane four neighbours of a group
  const int seg = ((r.padded >> 7) + kSmpWarps - 1) / kSmpWarps * 128;
  const int beg = min(r.padded, warp * seg), end = min(r.padded, beg + seg);
  const int draft_at = draft - r.begin;
  const bool open = BORDER && bd.open;
  u64 floor_key = !BORDER ? 0ull : open ? bd.floor : bd.key;
  float tau = floor_key ? smp_key_value(floor_key) : -INFINITY;
  int last = floor_key ? static_cast<int>(smp_id(floor_key)) - r.begin : 0x7fffffff;
  // kept: above the border's value, or at it and not behind its id
  auto keep = [&](float x, int i) { return !BORDER || x > tau || (x == tau && i <= last); };
  auto weight = [&](float x, int i) -> u64 { return keep(x, i) ? smp_weight(r, x) : 0ull; };
  if (open) {
    if (tid == 0) sh->n_own = 0;
    __syncthreads();
  }
  u64 mine = 0;
  if (r.fast) {
    for (int i0 = beg + lane * 4; i0 < end; i0 += 512) {
      float4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i0 + q * 128 < end) v[q] = smp_load4(r, i0 + q * 128);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + q * 128;
        if (i >= end) break;
        const float x[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
        u64 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = smp_bits(r, x[e]) - kSmpBias;
        if (r.w_min) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (w[e] < r.w_min) w[e] = 0;
        }
        if (open) {
          // what lies before the border's bin is kept; the bin's tokens are listed: the
          // ones that were counted there, which for weights leaves out those that
          // weigh nothing (under min_p, and many of them in a flat row)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int side = bd.bins.side(x[e], bd.bin);
            if (side != 0) w[e] = side < 0 ? w[e] : 0;
            else if ((w[e] || !bd.by_mass) && keep(x[e], i + e))
              smp_candidate(x[e], r.begin + i + e);
            if (side == 0) w[e] = 0;
          }
        } else if (BORDER) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!keep(x[e], i + e)) w[e] = 0;
        }
        mine += (w[0] + w[1]) + (w[2] + w[3]);
      }
    }
  } else {
    for (int i = beg + lane * 4; i < end; i += 128) {
      const float4 v = smp_load4(r, i);
      mine += weight(v.x, i) + weight(v.y, i + 1) + weight(v.z, i + 2) + weight(v.w, i + 3);
    }
  }
  if (open) {
    // the border among the listed tokens, and the kept ones' weights to their warps
    floor_key = smp_close(r, bd, bd.by_mass ? 1 : 0);
    tau = smp_key_value(floor_key);
    last = static_cast<int>(smp_id(floor_key)) - r.begin;
    unsigned* lo = sh->run_w[0];
    unsigned* hi = sh->run_w[1];
    if (tid < kSmpWarps) lo[tid] = hi[tid] = 0;
    __syncthreads();
    // (rank 0 searched in the place of its own list, but has everybody's)
    const u64* listed = r.rank == 0 ? sh->list : sh->own;
    const int n = min(r.rank == 0 ? sh->n_list[bd.by_mass ? 2 : 1] : sh->n_own,
                      static_cast<unsigned>(kSmpList));
    for (int c = tid; c < n; c += kSmpThreads) {
      const u64 key = listed[c];
      const int i = static_cast<int>(smp_id(key)) - r.begin;
      if (key < floor_key || i >= r.len) continue;
      smp_add(&lo[i / seg], &hi[i / seg], smp_weight(r, smp_key_value(key)));
    }
    __syncthreads();
    if (lane == 0) mine += lo[warp] + (static_cast<u64>(hi[warp]) << 32);
  }
  const u64 in_warp = warp_sum_u64(mine);
  const u64 upto = smp_block_scan(lane == 0 ? in_warp : 0ull);
  if (tid == kSmpThreads - 1) {
    const u64 d = draft >= 0 && draft_at >= 0 && draft_at < r.len
                      ? weight(__ldg(r.x + draft_at), draft_at)
                      : 0ull;
    for (int k = 0; k < kSmpRanks; ++k) {
      st_peer_u64(&sh->kept_in[r.rank], k, upto);
      st_peer_u64(&sh->draft_in[r.rank], k, d);
    }
  }
  if (tid == 0) sh->found = kSmpWarps;
  cluster_sync();   // the row's last: no CTA touches another's memory behind it
  u64 before = 0, total = 0, draft_w = 0;
  int draft_rank = -1;
  for (int k = 0; k < kSmpRanks; ++k) {
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
    sh->found = warp;
    sh->bcast[0] = run;
  }
  __syncthreads();
  if (sh->found >= kSmpWarps) return out;        // not in this slice
  // the CTA scans that run together, four neighbours a thread
  const int b0 = static_cast<int>(sh->found) * seg, b1 = min(r.padded, b0 + seg);
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

__device__ __noinline__ SmpResult smp_draw_bordered(const SmpRow r, const SmpBorder bd, int draft,
                                                    float u_accept, float u) {
  return smp_draw_row<true>(r, bd, draft, u_accept, u);
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
  SmpResult out = {0, 0, -1, 0.f};
  u64 floor_key = 0, before;
  for (int i = tid; i < n; i += kSmpThreads) sh->w[i] = 1;
  __syncthreads();
  if (k > 0 && k < n) {
    const int at = smp_cross(n, false, false, 0ull, static_cast<double>(k), &before);
    floor_key = at >= 0 ? sh->list[at] : 0ull;
  }
  u64 sum = 0;
  for (int i = tid; i < n; i += kSmpThreads) {
    const u64 w = sh->list[i] >= floor_key ? smp_weight(r, smp_key_value(sh->list[i])) : 0ull;
    sh->w[i] = w;
    sum += w;
  }
  sum = smp_block_sum(sum);
  const double goal = fmax(top_p * static_cast<double>(mass_all ? mass_all : sum), 1.0);
  if (goal <= static_cast<double>(sum)) {
    const int at = smp_cross(n, false, false, 0ull, goal, &before);
    if (at >= 0) floor_key = max(floor_key, sh->list[at]);
  }
  u64 draft_w = 0, total = 0;
  for (int i = tid; i < n; i += kSmpThreads) {
    u64 w = sh->w[i];
    if (sh->list[i] < floor_key) w = 0;
    if (static_cast<int>(smp_id(sh->list[i])) == draft) {
      draft_w = w;
      w = 0;
    }
    sh->w[i] = w;
    total += w;
  }
  total = smp_block_sum(total);             // without the draft
  draft_w = smp_block_sum(draft_w);
  if (smp_accepts(draft_w, total + draft_w, u_accept)) {
    out.writer = tid == 0;
    out.accepted = 1;
    out.token = draft;
    return out;
  }
  out.writer = tid == 0;
  if (total == 0) return out;
  const int at = smp_cross(n, true, true, 0ull,
                           static_cast<double>(smp_unit(u)) * static_cast<double>(total), &before);
  if (at >= 0) {
    out.token = static_cast<int>(smp_id(sh->list[at]));
    out.prob = smp_share(sh->w[at], total);
  }
  return out;
}

// One row: maxima, filters, draw.  Exactly one thread of the cluster returns with
// writer set.  Entered behind smp_arrive().
__device__ __forceinline__ SmpResult smp_row(const float* row, int V, int slice,
                                             const SampleSettings& set, int at, int draft,
                                             float u_accept, float u) {
  SmpShared* sh = smp_shared();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  SmpRow r;
  r.rank = static_cast<int>(cluster_rank());
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
  const float scale = fminf((kSmpMaxBins - 1) / (kSmpReach * T), 3e38f);
  const float fine = fminf((kSmpBins - 1) / (kSmpReach * T), 3e38f);
  const bool by_list = !greedy && by_k && k_in <= kSmpListTopK;
  if (!greedy) {
    for (int i = tid; i < kSmpTab; i += kSmpThreads) sh->tab[i] = exp2(kSmpOneBits + i * (1.0 / kSmpTab));
    if (by_list)
      for (int i = tid; i < kSmpMaxBins; i += kSmpThreads) sh->cnt[i] = 0;
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
    if (b < kSmpMaxBins) atomicAdd(&sh->cnt[b], 1u);
    __syncthreads();
    constexpr int kPer = kSmpMaxBins / kSmpThreads;
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
  smp_wait();
  if (tid < kSmpRanks) {
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
    top = lane < kSmpRanks ? sh->top_in[lane] : -INFINITY;
    if (by_list) {
      const float v = c < kSmpRanks ? sh->thr_in[c][j] : -INFINITY;
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
    for (int k = 0; k < kSmpRanks; ++k) id = min(id, sh->first_in[k]);
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
  if (!by_k && !by_p) return smp_draw_row<false>(r, smp_at_key(0ull), draft, u_accept, u);
  SmpBorder border = smp_at_key(0ull);
  u64 mass_all = 0;
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
    if (r.rank == 0 && tid < kSmpRanks) st_peer_u32(&sh->verdict, tid, sh->n_list[0] <= kSmpList);
    cluster_sync();
    listed = sh->verdict != 0;
  }
  if (!listed) {
    if (by_k) border = smp_border_k(r, fine, static_cast<u64>(k_in));
    if (by_p)
      border = smp_border_p(r, fine, by_k ? smp_resolve(r, border, 0) : 0ull, top_p, &listed,
                            &mass_all);
  }
  if (!listed) return smp_draw_bordered(r, border, draft, u_accept, u);
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
  smp_arrive();
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
};

// Cluster (y, z) settles row z of request y.  Clusters start in the order of z:
// when a late one starts, an earlier row of its request may have refused, and
// the row has nothing to say.  Whether it looks only decides if work is saved: a
// request's answer is its first refusing row's, whoever ran.  The cluster that
// settles a request's last row writes the answer.  (Runs of two, four or eight
// rows a cluster, which spare launches, took 1.3 to 1.5 times as long at 128
// requests of 16 rows: the rows of one request then wait in line.)
__global__ void __launch_bounds__(kSmpThreads, kSmpCtas)
verify_sampled_kernel(const VerifySampledParams p) {
  pdl_trigger();
  pdl_wait();
  SmpShared* sh = smp_shared();
  const int b = blockIdx.y, i = blockIdx.z, K = p.K;
  const bool lead = threadIdx.x == 0 && cluster_rank() == 0;
  bool needed = true;
  if (i > 0) {
    // one reading for the whole cluster: rank 0's
    if (lead) {
      const unsigned refused = *reinterpret_cast<volatile unsigned*>(p.refused + b);
      sh->more = !(refused && i > K + 1 - static_cast<int>(refused));
    }
    cluster_sync();
    needed = ld_peer_u32(&sh->more, 0) != 0;
  }
  if (needed) smp_arrive();
  else cluster_sync();       // rank 0 stays until every CTA has read its word
  if (needed) {
    const int draft = i < K ? p.drafts[static_cast<int64_t>(b) * K + i] : -1;
    const SmpResult res =
        smp_row(p.logits + (static_cast<int64_t>(b) * (K + 1) + i) * p.ld, p.V, p.slice, p.set, b,
                draft, i < K ? p.u_accept[static_cast<int64_t>(b) * K + i] : 0.f, p.u_sample[b]);
    if (!res.writer) return;
    if (!res.accepted || i == K) {
      p.row_token[static_cast<int64_t>(b) * (K + 1) + i] = res.token;
      __threadfence();
      atomicMax(p.refused + b, static_cast<unsigned>(K + 1 - i));
    }
  } else if (!lead) {
    return;
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
