// prefix_attention.cuh — attention of a batch of query blocks whose requests
// share their first pages.
//
// o = softmax(q K^T / sqrt(D)) V over the keys of a row is a sum over parts of
// them: with a reference m, l = sum 2^(s - m) and O = sum 2^(s - m) v of each
// part (s in units of log2), the whole is sum 2^(m - M) O / sum 2^(m - M) l.
// A part is left as (m, l, O / l) in fp32.  So the shared prefix is one dense
// attention of every row of the batch against keys that are read once, each
// request's own keys are another, and a merge joins them.
//   prefix   bound by the tensor cores: 6 D flops a row and key, the keys read
//            once per 256 rows from L2
//   own keys bound by HBM: 4 D bytes a key and kv head
// P is held as two bf16, the second what the first leaves, and multiplied with V
// twice (2^-15 of each weight; the 4 D flops of a formula become 6 D).  One bf16,
// and parts in fp16, leave eight times the error, 1.7e-3 of the result against
// 2.1e-4, the rounding of the output to fp16 (16, 134 and 447 us for calls of 16, 512
// and 1280 tokens that now take 18, 176 and 600).
//
// attn_part_kernel<D, NT, KT> runs both.  NT row tiles of 128 query rows share
// the K/V tiles of KT keys that pass through a ring in shared memory; S and,
// in its place, P (two bf16) stay in tensor memory beside O:
//   warp 0      TMA producer: lane j loads page j % (KT / 16), column half j / ..
//   warp 1      MMA issuer (one thread): S = Q K^T, O += P V with P read from
//               tensor memory
//   then 4 warps for each row tile: thread = row, so the maximum, the sum and
//               the mask of a row need no exchange
// NT = 2: the issue order PV_0(t) S_0(t+1) PV_1(t) S_1(t+1) keeps the tensor cores
// on one row tile while the other one's softmax runs.  NT = 1: S has two buffers,
// S(t+1) is issued before P V(t), and a second CTA on the SM fills the rest.
//
// Measured at 128 requests x 10 rows over 16384 shared keys (NT = 2): a pair of row
// tiles takes 5500 cycles a key tile, 3100 of them products; what is left is the chain
// S, softmax, P V of a row tile, whose softmax shares the exponential units with the
// other tile's (40 % busy).  With one bf16 a weight 4080 cycles, 2020 products.  Tried
// with that and slower: an issuer for each row tile (448 us against 347), eight
// softmax warps a row tile (357), a quarter or half of the exponentials as polynomials
// on the FMA pipes (347, 373).  With two, calls of 1280 tokens: handing P over in
// halves (617 us against 605), all high products before the low ones (598 and 596).
//   NT = 2, KT = 128: one CTA an SM, 256 flops of the formula per byte read, for
//                     many rows
//   NT = 1, KT = 64:  two CTAs an SM, for one request's rows
#pragma once

#include "dflash_device.cuh"

namespace dflash {

constexpr float kPartHeadroom = 32.f;   // log2 of the largest 2^(s - m) kept unscaled

struct PartParams {
  // query tokens [n_tok = B * q_len][Hq][D]; row r of a tile that starts at
  // token t: token t + r / G, query head h * G + r % G
  int B, q_len, n_tok, Hq, Hkv, G, tpt;   // tpt = 128 / G tokens a tile
  int causal;
  const bf16 *q, *k_cache, *v_cache;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int W, num_pages, prefix_keys;
  // the prefix, dealt to the first prefix_ctas CTAs in equal runs of
  // (item = kv head and row tiles, key tile)
  int prefix_ctas, prefix_items, prefix_tiles, row_groups;   // row_groups = items per kv head
  unsigned prefix_run;   // units of a CTA; all units fit 31 bits
  int max_segs;
  float* prefix_o;     // [prefix_ctas][max_segs][NT][128][D]
  float2* prefix_ml;   // [prefix_ctas][max_segs][NT][128]
  // own keys: one CTA a (split, request, kv head)
  int chunk_keys, max_splits, R;          // R = q_len * G
  float* own_o;        // [max_splits][B][Hkv][R][D]
  float2* own_ml;      // [max_splits][B][Hkv][R]
  float scale_log2;
  unsigned* err;
};

template <int D_, int NT_, int KT_>
struct PartCfg {
  static constexpr int D = D_, NT = NT_, KT = KT_;
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = KT * D * 2;
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kCtas = NT == 1 ? 2 : 1;            // per SM
  static constexpr int kRoom = 232448 / kCtas - 2048;
  static constexpr int kFit = (kRoom - NT * kQBytes) / kTileBytes;
  static constexpr int NS = kFit > 6 ? 6 : kFit;           // ring slots (K or V tiles)
  static constexpr int kOffRing = NT * kQBytes;
  static constexpr int kOffBar = kOffRing + NS * kTileBytes;
  static constexpr int kSmem = 1024 + kOffBar + 256;
  static constexpr int kThreads = 64 + NT * 128;
  static constexpr int kUsed = 2 * KT + NT * D;            // S twice, O
  static constexpr int kCols = kUsed > 256 ? 512 : kUsed > 128 ? 256 : 128;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(NS >= 3, "ring");
  static_assert(kCols * kCtas <= 512, "tensor memory");
};

__device__ __forceinline__ float part_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void part_fence_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void part_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                             int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// D[tmem] (+)= A * B[smem]^T, bf16 inputs; A in shared memory, or in tensor memory
// as 128 lanes x packed pairs.  One thread issues every product, and an operation
// of one thread takes several cycles while a 128 x 128 x 16 product takes 64: so
// a descriptor is one addition to its low word, and what is constant is an
// immediate.
template <bool ACC>
__device__ __forceinline__ void part_mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi,
                                            uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void part_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void part_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// kind::f16, bf16 x bf16 -> fp32; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t part_idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Column of the weights of keys 16 kk .. 16 kk + 15 of a tile, high halves; the low
// ones are 16 columns on.
__device__ __forceinline__ constexpr int part_p_at(int kk) { return (kk >> 1) * 32 + (kk & 1) * 8; }

// Two floats in a 64-bit register: the FMA pipes take both in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 part_pack(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void part_unpack(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 part_fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 part_add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Two floats as bf16, rounded towards zero (lo in the low half).
__device__ __forceinline__ uint32_t part_cut_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float part_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// P = 2^(s scale - ref) in the place of KT of a row's scores; returns their sum.  Chunk
// c of 32 scores is read from columns 32 c .. and gives its place to the bf16 pairs
// of P, and behind them (part_p_at) those of what they leave.  The first is cut off, not
// rounded, and 2^-20 of it is added to the second: both halves of a weight above 0 are
// above 0, and an infinite V gives what it gives in the formula.
template <int KT, bool MASKED>
__device__ __forceinline__ float part_weights(uint32_t s_at, float scale, float ref, int left) {
  const f32x2 sc2 = part_pack(scale, scale), nr2 = part_pack(-ref, -ref);
  constexpr float kBelow = -1.f + 1.f / (1 << 20);
  const f32x2 minus = part_pack(kBelow, kBelow);
  f32x2 l2[2] = {part_pack(0.f, 0.f), part_pack(0.f, 0.f)};
  float x[2][32];
  tmem_ld_32x32b_x32(s_at, x[0]);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < KT / 32; ++c) {
    if (c + 1 < KT / 32) tmem_ld_32x32b_x32(s_at + (c + 1) * 32, x[(c + 1) & 1]);
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a = x[c & 1][2 * e], b = x[c & 1][2 * e + 1];
      if (MASKED) {
        if (c * 32 + 2 * e >= left) a = -INFINITY;
        if (c * 32 + 2 * e + 1 >= left) b = -INFINITY;
      }
      const f32x2 y = part_fma2(part_pack(a, b), sc2, nr2);
      part_unpack(y, a, b);
      a = part_ex2(a);
      b = part_ex2(b);
      l2[e & 1] = part_add2(l2[e & 1], part_pack(a, b));
      w[e] = part_cut_bf16x2(a, b);
      part_unpack(part_fma2(part_pack(__uint_as_float(w[e] << 16),
                                      __uint_as_float(w[e] & 0xffff0000u)),
                            minus, part_pack(a, b)),
                  a, b);
      w[16 + e] = pack_bf16x2(a, b);
    }
    if (c + 1 < KT / 32) tmem_ld_wait();
    part_st_x32(s_at + c * 32, w);
  }
  float la, lb;
  part_unpack(part_add2(l2[0], l2[1]), la, lb);
  return la + lb;
}

// One run of key tiles for one set of row tiles.
struct PartSeg {
  int h, tok0, b;      // b: whose table row and own keys; -1: the prefix
  int key0, key1;      // absolute keys, key0 a multiple of 16
  int n_tiles;
  int slot;            // partial result
};

// The CTA's segments in turn; every role of the CTA walks them alike.
template <int NT, int KT>
struct PartWalk {
  int next = 0;       // next one to look at
  __device__ __forceinline__ bool step(const PartParams& p, PartSeg& s) {
    if (static_cast<int>(blockIdx.x) < p.prefix_ctas) {
      // CTA c has the (item, tile) units [c * run, (c + 1) * run)
      const unsigned u0 = blockIdx.x * p.prefix_run;
      const unsigned u1 = min(u0 + p.prefix_run,
                              static_cast<unsigned>(p.prefix_items) * p.prefix_tiles);
      const unsigned item = u0 / p.prefix_tiles + next;
      const unsigned first = item * p.prefix_tiles;
      const unsigned a = max(u0, first), e = min(u1, first + p.prefix_tiles);
      if (first >= u1 || a >= e) return false;
      const int t0 = static_cast<int>(a - first);
      s.n_tiles = static_cast<int>(e - a);
      s.h = item / p.row_groups;
      s.tok0 = (item - s.h * p.row_groups) * NT * p.tpt;
      s.b = -1;
      s.key0 = t0 * KT;
      s.key1 = min(p.prefix_keys, (t0 + s.n_tiles) * KT);
      s.slot = blockIdx.x * p.max_segs + next;
      ++next;
      return true;
    }
    if (next++ > 0) return false;
    // own keys: one item (split, request, kv head), the kv head fastest
    const int i = static_cast<int>(blockIdx.x) - p.prefix_ctas;
    const int rest = i / p.Hkv, split = rest / p.B;
    s.b = rest - split * p.B;
    const int seq = p.seq_lens[s.b];
    s.key0 = p.prefix_keys + split * p.chunk_keys;
    // 64-bit: seq may be anything
    s.key1 = seq < 0 ? 0
                     : static_cast<int>(min(static_cast<long long>(seq) + p.q_len,
                                            static_cast<long long>(s.key0) + p.chunk_keys));
    s.h = i - rest * p.Hkv;
    s.n_tiles = (s.key1 - s.key0 + KT - 1) / KT;
    s.tok0 = s.b * p.q_len;
    s.slot = i;
    return s.key0 < s.key1;
  }
};

template <int D, int NT, int KT>
__global__ void __launch_bounds__(PartCfg<D, NT, KT>::kThreads, NT == 1 ? 2 : 1)
attn_part_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const PartParams p) {
  using C = PartCfg<D, NT, KT>;
  constexpr int NS = C::NS, kHalves = C::kHalves;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PartSeg seg;
  PartWalk<NT, KT> walk;
  if (!walk.step(p, seg)) return;   // the same for the whole CTA
  constexpr int kPages = KT / 16;
  const int pj = lane % kPages, half = lane / kPages;   // a producer lane's page and column half
  // row of the pools' [pages * Hkv * 16, D] view where this lane's page of tile t
  // starts; -16 (zeros are filled in) past the range, the table or the pool
  auto page_row = [&](int t) {
    const int key = seg.key0 + t * KT + pj * 16;
    if (t >= seg.n_tiles || key >= seg.key1) return -16;
    const int pg = key >> 4;
    if (pg >= p.W) {
      raise_error(p.err, DFLASH_DEVERR_TABLE);
      return -16;
    }
    const int page = p.block_table[static_cast<size_t>(max(seg.b, 0)) * p.W + pg];
    if (page < 0 || page >= p.num_pages) {
      raise_error(p.err, DFLASH_DEVERR_SLOT);
      return -16;
    }
    return (page * p.Hkv + seg.h) * 16;
  };
  // the first pages' numbers come while the CTA sets itself up
  int row = -16, next_row = -16;
  if (warp == 0) {
    row = page_row(0);
    next_row = page_row(1);
  }
  extern __shared__ uint8_t part_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(part_smem) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* full = bars;             // [NS] a K or V tile has landed
  uint64_t* empty = bars + 8;        // [NS] its last MMA has run
  uint64_t* q_full = bars + 16;
  uint64_t* q_empty = bars + 17;     // the segment's last S has run
  // S buffer: row tile i (NT = 2), or key tile % 2 (NT = 1)
  uint64_t* s_full = bars + 18;      // [2] S of a tile is there
  uint64_t* p_full = bars + 20;      // [2] P of a tile is written
  uint64_t* o_full = bars + 22;      // [NT] the segment's last P V has run
  uint64_t* o_free = bars + 24;      // [NT] O has been read
  uint64_t* pv_done = bars + 26;     // NT = 1: P V of a tile has run
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 27);
  auto ring = [&](int s) { return smem + C::kOffRing + s * C::kTileBytes; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 4);
    }
    mbar_init(pv_done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto col_s = [&](int buf) { return tmem + buf * KT; };
  auto col_o = [&](int i) { return tmem + 2 * KT + i * D; };
  // phase of an S buffer's barriers for the CTA's n-th key tile
  auto s_buf = [&](int i, unsigned n) { return NT == 2 ? i : static_cast<int>(n & 1); };
  auto s_phase = [&](unsigned n) { return (NT == 2 ? n : n >> 1) & 1u; };
  // The ring holds K_0, then K_(t+1), V_t for each t: the order of use.
  // K_t is tile 2t - 1 of its segment (K_0: 0), V_t tile 2t + 2 (the last: 2t + 1).

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const bool loads = lane < kPages * kHalves;
    unsigned seq = 0;      // ring tiles issued
    unsigned q_loads = 0;
    bool ok = true, more = true;
    for (int k = 0; ok && more; ++k) {
      if (k > 0) {
        row = page_row(0);
        next_row = page_row(1);
      }
      if (lane == 0) {
        ok = mbar_wait(q_empty, (k & 1) ^ 1u, p.err);
        if (ok) {
          mbar_arrive_expect_tx(q_full, NT * kHalves * p.tpt * p.G * 128);
          for (int i = 0; i < NT; ++i)
            for (int hf = 0; hf < kHalves; ++hf)
              part_load_3d(smem + (i * kHalves + hf) * 128 * 128, &tmQ, q_full, hf * 64,
                           seg.h * p.G, seg.tok0 + i * p.tpt);
          ++q_loads;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      auto issue = [&](const CUtensorMap* map, int at) {
        const int s = seq % NS;
        if (lane == 0) {
          ok = mbar_wait(&empty[s], ((seq / NS) & 1) ^ 1u, p.err);
          if (ok) mbar_arrive_expect_tx(&full[s], C::kTileBytes);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        __syncwarp();
        if (ok && loads)
          tma_load_2d(ring(s) + half * KT * 128 + pj * 2048, map, &full[s], half * 64, at);
        ++seq;
      };
      if (ok) issue(&tmK, row);
      for (int t = 0; ok && t < seg.n_tiles; ++t) {
        const int after = page_row(t + 2);
        if (t + 1 < seg.n_tiles) issue(&tmK, next_row);
        if (ok) issue(&tmV, row);
        row = next_row;
        next_row = after;
      }
      more = walk.step(p, seg);
    }
    if (!ok && lane == 0) {
      // given up: let the copies in flight land before the CTA's memory goes
      for (int spin = 0;
           q_loads && spin < 100000 && !mbar_test_wait(q_full, (q_loads - 1) & 1); ++spin) {
      }
      for (unsigned s = seq > NS ? seq - NS : 0; s < seq; ++s)
        for (int spin = 0; spin < 100000 && !mbar_test_wait(&full[s % NS], (s / NS) & 1); ++spin) {
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = part_idesc(128, KT, false);
      constexpr uint32_t id_o = part_idesc(128, D, true);
      const uint64_t dq = umma_desc_sw128(smem_u32(smem));
      const uint64_t dk = umma_desc_sw128(smem_u32(ring(0)));
      const uint64_t dv = umma_desc_sw128_mn(smem_u32(ring(0)), KT * 128, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
      constexpr uint32_t kSlot = C::kTileBytes >> 4;     // addresses count 16 bytes
      unsigned tiles = 0;                 // key tiles done before this segment
      unsigned slot = 0, wraps = 0;       // of the next ring tile
      bool ok = true;
      auto advance = [&]() {
        if (++slot == NS) {
          slot = 0;
          ++wraps;
        }
      };
      auto mma_s = [&](int i, int buf, uint32_t k_at) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int hf = kk >> 2, w = kk & 3;
          const uint32_t qa = q_lo + (i * kHalves + hf) * (128 * 128 / 16) + w * 2;
          const uint32_t ka = k_at + hf * (KT * 128 / 16) + w * 2;
          if (kk == 0) part_mma_ss<false>(col_s(buf), qa, q_hi, ka, k_hi, id_s);
          else part_mma_ss<true>(col_s(buf), qa, q_hi, ka, k_hi, id_s);
        }
        umma_commit(&s_full[buf]);
      };
      bool more_segs = true;
      for (int k = 0; ok && more_segs; ++k, more_segs = walk.step(p, seg)) {
        const int n_tiles = seg.n_tiles;
        ok = mbar_wait(q_full, k & 1, p.err) && mbar_wait(&full[slot], wraps & 1, p.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < NT; ++i) mma_s(i, s_buf(i, tiles), k_lo + slot * kSlot);
        umma_commit(&empty[slot]);
        if (n_tiles == 1) umma_commit(q_empty);
        advance();
        for (int t = 0; ok && t < n_tiles; ++t) {
          const bool more = t + 1 < n_tiles;
          const unsigned n = tiles + t, kslot = slot;
          // K of the next tile lies before V of this one in the ring
          if (more) {
            ok = mbar_wait(&full[kslot], wraps & 1, p.err);
            advance();
            if (NT == 1 && ok) {
              // the other S buffer's P was read by the P V issued before
              tc_fence_after();
              mma_s(0, s_buf(0, n + 1), k_lo + kslot * kSlot);
              umma_commit(&empty[kslot]);
              if (t + 2 == n_tiles) umma_commit(q_empty);
            }
          }
          if (ok) ok = mbar_wait(&full[slot], wraps & 1, p.err);
          const uint32_t v_at = v_lo + slot * kSlot;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const int buf = s_buf(i, n);
            // the first P V of a segment overwrites O: the last one's must be read
            if (ok && t == 0) ok = mbar_wait(&o_free[i], (k & 1) ^ 1u, p.err);
            if (ok) ok = mbar_wait(&p_full[buf], s_phase(n), p.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
              const uint32_t p_at = col_s(buf) + part_p_at(kk), v_kk = v_at + kk * (16 * 128 / 16);
              part_mma_ts(col_o(i), p_at, v_kk, v_hi, id_o, kk > 0 || t > 0 ? 1u : 0u);
              part_mma_ts(col_o(i), p_at + 16, v_kk, v_hi, id_o, 1u);
            }
            if (NT == 1) umma_commit(pv_done);
            if (!more) umma_commit(&o_full[i]);
            if (NT == 2 && more) mma_s(i, buf, k_lo + kslot * kSlot);
          }
          if (!ok) break;
          if (NT == 2 && more) {
            umma_commit(&empty[kslot]);
            if (t + 2 == n_tiles) umma_commit(q_empty);
          }
          umma_commit(&empty[slot]);
          advance();
        }
        tiles += n_tiles;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int i = (warp - 2) >> 2;                   // row tile
    const int sp = warp & 3;                         // tensor-memory sub-partition
    const int r = 32 * sp + lane;                    // row of the tile
    const uint32_t lanes = static_cast<uint32_t>(32 * sp) << 16;
    const float scale = p.scale_log2;
    unsigned tiles = 0, seq = 0;
    bool ok = true;
    bool more = true;
    for (int k = 0; more; ++k, more = walk.step(p, seg)) {
      // keys that this row sees: none if it is no row of this segment
      int limit = 0;
      {
        const int tr = r / p.G;
        const int tok = seg.tok0 + i * p.tpt + tr;
        if (tr < p.tpt && tok < p.n_tok) {
          const int b = tok / p.q_len, j = tok - b * p.q_len;
          const int n = p.seq_lens[b];
          if ((seg.b < 0 || seg.b == b) && n >= 0)
            limit = static_cast<int>(min(static_cast<long long>(n) + (p.causal ? j + 1 : p.q_len),
                                         static_cast<long long>(seg.key1)));
        }
      }
      // a warp without rows only keeps step: its P and O rows are never stored
      const bool rows = __any_sync(0xffffffffu, limit > seg.key0);
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < seg.n_tiles; ++t) {
        const unsigned n = tiles + t;
        const int buf = s_buf(i, n);
        if (ok) ok = mbar_wait(&s_full[buf], s_phase(n), p.err);
        tc_fence_after();
        if (rows) {
          const uint32_t s_at = col_s(buf) + lanes;
          const int left = limit - (seg.key0 + t * KT);    // keys of the tile that the row sees
          // (a CTA of one row tile lives for a few tiles, and its code comes from L2:
          // one path is quicker than two, 16 single tokens 17.8 us against 19.9)
          const bool masked = NT == 1 || __any_sync(0xffffffffu, left < KT);
          float mx;
          {
            // S is read twice, for the maximum and for P: the second reading costs
            // less than the registers that a row of it would hold meanwhile
            float x[KT];
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) tmem_ld_32x32b_x32(s_at + c * 32, x + c * 32);
            tmem_ld_wait();
            if (masked) {
#pragma unroll
              for (int c = 0; c < KT; ++c)
                if (c >= left) x[c] = -INFINITY;
            }
            float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c + 8 <= KT; c += 8) {
#pragma unroll
              for (int e = 0; e < 4; ++e) mx4[e] = part_max3(mx4[e], x[c + e], x[c + 4 + e]);
            }
            mx = part_max3(part_max3(mx4[0], mx4[1], x[KT - 4]),
                           part_max3(mx4[2], mx4[3], x[KT - 3]),
                           fmaxf(x[KT - 2], x[KT - 1])) * scale;
          }
          // The reference is the first maximum that the row meets; it is raised only
          // when a score outgrows it by the headroom (2^32 keeps P, l and O far inside
          // their types), so O is rarely rescaled.
          if (__any_sync(0xffffffffu, mx > m + kPartHeadroom)) {
            const float up = mx > m + kPartHeadroom ? mx : m;
            const float a = m == -INFINITY ? 0.f : part_ex2(m - up);
            const bool has = __any_sync(0xffffffffu, m != -INFINITY);
            m = up;
            l *= a;
            if (has && t > 0) {
              // P V of the tile before must have run: with NT = 2 s_full came after it
              if (NT == 1) {
                if (ok) ok = mbar_wait(pv_done, (n - 1) & 1u, p.err);
                tc_fence_after();
              }
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld_32x32b_x32(col_o(i) + lanes + c * 32, o);
                tmem_ld_wait();
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * a);
                part_st_x32(col_o(i) + lanes + c * 32, w);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          l += masked ? part_weights<KT, true>(s_at, scale, ref, left)
                      : part_weights<KT, false>(s_at, scale, ref, left);
        }
        if (NT == 1 && sp == 0 && t + 1 == seg.n_tiles && (seg.key1 & 15)) {
          // rows of V past the last key of its page may hold anything (NaN too):
          // zeros there, so that P = 0 adds 0
          const unsigned vq = seq + 2 * seg.n_tiles - 1;
          if (ok) ok = mbar_wait(&full[vq % NS], (vq / NS) & 1, p.err);
          const int end = seg.key1 - (seg.key0 + t * KT);
          const int n16 = (16 - (end & 15)) * kHalves * 8;
          for (int e = lane; e < n16; e += 32) {
            const int hf = e & (kHalves - 1), cc = (e / kHalves) & 7, rr = end + e / (kHalves * 8);
            *reinterpret_cast<uint4*>(ring(vq % NS) + hf * KT * 128 + rr * 128 + cc * 16) =
                make_uint4(0, 0, 0, 0);
          }
          part_fence_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      // the part: O, and (m, l) of the row
      if (ok) ok = mbar_wait(&o_full[i], k & 1, p.err);
      tc_fence_after();
      const bool own = seg.b >= 0;
      float* dst = own ? p.own_o + (static_cast<size_t>(seg.slot) * p.R + r) * D
                       : p.prefix_o + ((static_cast<size_t>(seg.slot) * NT + i) * 128 + r) * D;
      const bool store = ok && rows && l != 0.f &&   // a NaN is a result
                         (!own || r < p.R);
      const float inv = 1.f / l;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        if (!rows) break;
        float o[32];
        tmem_ld_32x32b_x32(col_o(i) + lanes + c * 32, o);
        tmem_ld_wait();
        if (store) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(dst + c * 32 + e) =
                make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
        }
      }
      const float2 stats = make_float2(m, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[i]);
      if (own) {
        if (r < p.R) p.own_ml[static_cast<size_t>(seg.slot) * p.R + r] = stats;
      } else {
        p.prefix_ml[(static_cast<size_t>(seg.slot) * NT + i) * 128 + r] = stats;
      }
      tiles += seg.n_tiles;
      seq += 2 * seg.n_tiles;
    }
  }
  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// A row whose result is not finite though keys are masked for it: P = 0 times a
// masked V that is not finite leaves NaN in the product.  If there is such a V,
// the row is summed again over the keys [0, limit) alone; only broken values reach this, so it is plain: one key a step.
// The lanes of a head (D / 8, eight dims each) work together.
template <int D>
__device__ __noinline__ void attn_row_again(const PartParams& p, int tok, int b, int h, int head,
                                            int limit, int end, int c8, float* out) {
  auto row_of = [&](int key) -> int64_t {
    const int pg = key >> 4;
    if (pg >= p.W) return -1;
    const bool shared = key < p.prefix_keys;
    const int page = p.block_table[static_cast<size_t>(shared ? 0 : b) * p.W + pg];
    if (page < 0 || page >= p.num_pages) return -1;
    return ((static_cast<int64_t>(page) * p.Hkv + h) * 16 + (key & 15)) * D + c8;
  };
  auto load8 = [](const bf16* src, float* x) {
    const uint4 w = *reinterpret_cast<const uint4*>(src);
    const __nv_bfloat162* t = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 f = __bfloat1622float2(t[c]);
      x[2 * c] = f.x;
      x[2 * c + 1] = f.y;
    }
  };
  float x[8], qv[8], acc[8];
  bool bad = false;
  for (int key = limit; key < end; ++key) {
    const int64_t at = row_of(key);
    if (at < 0) continue;
    load8(p.v_cache + at, x);
#pragma unroll
    for (int c = 0; c < 8; ++c) bad |= !(fabsf(x[c]) <= 3.4e38f);
  }
  if (!__any_sync(0xffffffffu, bad)) return;      // the row's own result
  load8(p.q + (static_cast<int64_t>(tok) * p.Hq + head) * D + c8, qv);
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int key = 0; key < limit; ++key) {
    const int64_t at = row_of(key);
    float s = 0.f;
    if (at >= 0) {
      load8(p.k_cache + at, x);
#pragma unroll
      for (int c = 0; c < 8; ++c) s += qv[c] * x[c];
    }
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2;
    const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top;
    const float keep = m == -INFINITY ? 0.f : part_ex2(m - ref), w = part_ex2(s - ref);
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= keep;
    if (at >= 0) {
      load8(p.v_cache + at, x);
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += w * x[c];
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) out[c] = acc[c] * inv;
}

// One warp joins the parts of `heads` query heads of a token's kv group (all of
// them, or one where there are few tokens and many parts); prefix_nt: the row
// tiles of the kernel that ran the prefix.  A lane has eight dims of a head (16
// bytes of a part's row), so a warp has 256 / D heads at once, or as many shares of
// one head's parts; the loads of four parts are in flight before the first is used.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ PartParams p,
                                                        int prefix_nt, int heads,
                                                        f16* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  const int unit = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int per_tok = p.Hq / heads;
  if (unit >= p.n_tok * per_tok) return;
  const int tok = unit / per_tok, head0 = (unit - tok * per_tok) * heads;
  const int h = head0 / p.G, g0 = head0 - h * p.G;
  const int b = tok / p.q_len, j = tok - b * p.q_len;
  const int seq = p.seq_lens[b];
  if (seq < 0) return;                       // a padding request keeps its rows
  // parts: the prefix CTAs c0 .. that ran this item, then the own splits
  unsigned c0 = 0, item = 0;
  int n_prefix = 0, in_item = 0;
  if (p.prefix_ctas > 0) {
    const int tile = tok / p.tpt, rg = tile / prefix_nt;
    item = h * p.row_groups + rg;
    in_item = (tile - rg * prefix_nt) * 128 + (tok - tile * p.tpt) * p.G;
    c0 = item * p.prefix_tiles / p.prefix_run;
    n_prefix = ((item + 1) * p.prefix_tiles - 1) / p.prefix_run - c0 + 1;
  }
  const long long own = static_cast<long long>(seq) + p.q_len - p.prefix_keys;
  if (own > static_cast<long long>(p.W) * 16 - p.prefix_keys && lane == 0 && j == 0 && head0 == 0)
    raise_error(p.err, DFLASH_DEVERR_TABLE);
  const int n_own = own <= 0 || p.max_splits == 0
                        ? 0
                        : static_cast<int>(min(static_cast<long long>(p.max_splits),
                                               (own + p.chunk_keys - 1) / p.chunk_keys));
  const int parts = n_prefix + n_own;
  // where part q's rows of this group are
  auto at = [&](int q) -> size_t {
    if (q < n_prefix) {
      const unsigned c = c0 + q;
      const unsigned k = item - c * p.prefix_run / p.prefix_tiles;
      return (static_cast<size_t>(c) * p.max_segs + k) * prefix_nt * 128 + in_item;
    }
    return ((static_cast<size_t>(q - n_prefix) * p.B + b) * p.Hkv + h) * p.R + j * p.G;
  };
  // keys that this token sees, and the end of what its parts multiplied
  const long long all = static_cast<long long>(seq) + p.q_len;
  const int limit = static_cast<int>(min(all - (p.causal ? p.q_len - j - 1 : 0),
                                         static_cast<long long>(p.W) * 16));
  const int end = static_cast<int>(max(min(all, static_cast<long long>(p.W) * 16),
                                       static_cast<long long>(n_prefix ? p.prefix_keys : 0)));
  const int c8 = lane % kLanes * 8;
  f16* dst = out + (static_cast<size_t>(tok) * p.Hq + h * p.G) * D + c8;
  // one head: the lane groups take its parts in turn
  const int share = heads == 1 ? kAtOnce : 1, mine = heads == 1 ? lane / kLanes : 0;
  for (int gb = g0; gb < g0 + heads; gb += kAtOnce) {
    const int g = min(gb + lane / kLanes, g0 + heads - 1);
    float M = -INFINITY, l = 0.f, acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = 0.f;
    for (int q0 = mine; q0 < parts; q0 += 4 * share) {
      float2 ml[4];
      float4 o[4][2];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int q = min(q0 + s * share, parts - 1);
        const size_t row = at(q) + g;
        ml[s] = (q < n_prefix ? p.prefix_ml : p.own_ml)[row];
        // (a part that saw no key left no row: what is read there is not used)
        const float4* src = reinterpret_cast<const float4*>(
            (q < n_prefix ? p.prefix_o : p.own_o) + row * D + c8);
        o[s][0] = src[0];
        o[s][1] = src[1];
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (q0 + s * share >= parts || ml[s].y == 0.f) continue;
        const float top = fmaxf(M, ml[s].x);
        const float keep = M == -INFINITY ? 0.f : part_ex2(M - top);
        // (a part whose l is NaN keeps its weight whatever its reference)
        const float w = ml[s].y * (ml[s].x == -INFINITY ? 1.f : part_ex2(ml[s].x - top));
        M = top;
        l = l * keep + w;
        const float* v = reinterpret_cast<const float*>(o[s]);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = acc[c] * keep + v[c] * w;
      }
    }
    if (share > 1) {
#pragma unroll
      for (int s = kLanes; s < 32; s <<= 1) {
        const float M2 = __shfl_xor_sync(0xffffffffu, M, s);
        const float l2 = __shfl_xor_sync(0xffffffffu, l, s), top = fmaxf(M, M2);
        // (nothing seen, or an l that is NaN: the factor is 1)
        const float a = M == -INFINITY ? 1.f : part_ex2(M - top);
        const float b2 = M2 == -INFINITY ? 1.f : part_ex2(M2 - top);
        M = top;
        l = l * a + l2 * b2;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          acc[c] = acc[c] * a + __shfl_xor_sync(0xffffffffu, acc[c], s) * b2;
      }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    float sum = 0.f;                          // not finite if a value is not
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      acc[c] *= inv;
      sum += fabsf(acc[c]);
    }
    if (limit < end && __any_sync(0xffffffffu, !(sum <= 3.4e38f))) {
      float again[8];                         // (acc itself stays in registers)
#pragma unroll
      for (int c = 0; c < 8; ++c) again[c] = acc[c];
      attn_row_again<D>(p, tok, b, h, h * p.G + g, limit, end, c8, again);
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = again[c];
    }
    if (gb + lane / kLanes < g0 + heads) {
      uint4 w;
      w.x = pack_f16x2(acc[0], acc[1]);
      w.y = pack_f16x2(acc[2], acc[3]);
      w.z = pack_f16x2(acc[4], acc[5]);
      w.w = pack_f16x2(acc[6], acc[7]);
      *reinterpret_cast<uint4*>(dst + static_cast<size_t>(g) * D) = w;
    }
  }
}

}  // namespace dflash
