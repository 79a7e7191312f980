// append_kv.cuh — keys, values and queries that the caller projected itself:
// optional per-head RMSNorm, rotation by the handle's table, paged scatter.
#pragma once

#include "dflash_device.cuh"

namespace dflash {

struct AppendParams {
  const bf16 *k, *v, *q;                    // rows of [heads][D], row strides in elements
  int64_t k_stride, v_stride, q_stride;
  const bf16 *k_norm, *q_norm;              // [D] or null
  const int64_t *positions, *slots;
  int n, num_pages, Hq, Hkv, page_size, max_position;
  float eps;
  const float2* rope;                       // [max_position][D / 2] (cos, sin)
  bf16 *k_cache, *v_cache, *q_out;
  unsigned* err;
};

// For a row at position p and slot s, per head x of D elements with x' = x or
// x' = x * rsqrt(mean(x^2) + eps) * w:
//   k, q:  y[i]       = x'[i] cos(p f_i) - x'[i + D/2] sin(p f_i)
//          y[i + D/2] = x'[i + D/2] cos(p f_i) + x'[i] sin(p f_i)
//   v:     copied
// in fp32, rounded to bf16 once at the store (the type the caches hold).
// A lane owns the eight pairs (i .. i+7, i+D/2 ..), so D/16 lanes hold a head,
// a norm needs no more than their shuffles, and every access is 16 bytes.  A
// warp takes U heads for each of its 512/D lane groups from one row: the
// row's cos/sin are read once for all of them and 2U loads are in flight a lane.
// Memory bound: reads and writes 4 D bytes a head.  Measured: 32768 rows of 16
// heads of 128 take 61 us, 4.6 TB/s of the 6.5 that a copy reaches (a row's heads
// lie in as many pages' places, so the stores are pieces of 256 bytes); 2048 rows
// of 48 heads 16 us (floor 7); one row is the host's call.
template <int D, int U>
__global__ void __launch_bounds__(256) append_kv_kernel(const AppendParams p) {
  constexpr int kLanes = D / 16;            // lanes of a head
  constexpr int kGroups = 32 / kLanes;      // heads a warp holds at once
  constexpr int kHeads = kGroups * U;       // heads of a unit
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int i0 = (lane % kLanes) * 8;       // the lane's first pair
  const int group = lane / kLanes;
  const int heads = 2 * p.Hkv + (p.q ? p.Hq : 0);
  const int segs = (heads + kHeads - 1) / kHeads;
  const int64_t units = static_cast<int64_t>(p.n) * segs;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
       unit < units; unit += stride) {
    const int64_t row = unit / segs;
    const int seg = static_cast<int>(unit - row * segs);
    const int64_t slot = p.slots[row];
    const int64_t pos = p.positions[row];
    if (slot < 0) continue;                 // a padding row
    const int64_t page = slot / p.page_size;
    const int off = static_cast<int>(slot - page * p.page_size);
    if (page >= p.num_pages || pos < 0 || pos >= p.max_position) {
      if (seg == 0 && lane == 0)
        raise_error(p.err, page >= p.num_pages ? DFLASH_DEVERR_SLOT : DFLASH_DEVERR_POSITION);
      continue;
    }
    uint4 lo[U], hi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = seg * kHeads + u * kGroups + group;
      if (h >= heads) continue;
      const bf16* x;
      if (h < p.Hkv) x = p.k + row * p.k_stride + h * D;
      else if (h < 2 * p.Hkv) x = p.v + row * p.v_stride + (h - p.Hkv) * D;
      else x = p.q + row * p.q_stride + (h - 2 * p.Hkv) * D;
      lo[u] = *reinterpret_cast<const uint4*>(x + i0);
      hi[u] = *reinterpret_cast<const uint4*>(x + i0 + D / 2);
    }
    float c[8], s[8];
    const float4* rt = reinterpret_cast<const float4*>(p.rope + pos * (D / 2) + i0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = __ldg(rt + j);
      c[2 * j] = t.x;
      s[2 * j] = t.y;
      c[2 * j + 1] = t.z;
      s[2 * j + 1] = t.w;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = seg * kHeads + u * kGroups + group;
      const bool in = h < heads;
      const bool is_v = h >= p.Hkv && h < 2 * p.Hkv;
      const bool is_q = h >= 2 * p.Hkv;
      const bf16* w = is_q ? p.q_norm : p.k_norm;
      float a[8], b[8];
      const bf16* la = reinterpret_cast<const bf16*>(&lo[u]);
      const bf16* lb = reinterpret_cast<const bf16*>(&hi[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = in ? bf2f(la[j]) : 0.f;
        b[j] = in ? bf2f(lb[j]) : 0.f;
      }
      if (p.k_norm || p.q_norm) {           // the same for the whole launch
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += a[j] * a[j] + b[j] * b[j];
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (w && !is_v) {
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const uint4 wl = __ldg(reinterpret_cast<const uint4*>(w + i0));
          const uint4 wh = __ldg(reinterpret_cast<const uint4*>(w + i0 + D / 2));
          const bf16* wa = reinterpret_cast<const bf16*>(&wl);
          const bf16* wb = reinterpret_cast<const bf16*>(&wh);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a[j] *= r * bf2f(wa[j]);
            b[j] *= r * bf2f(wb[j]);
          }
        }
      }
      if (!in) continue;
      uint4 ya, yb;
      if (is_v) {
        ya = lo[u];
        yb = hi[u];
      } else {
        uint32_t* oa = reinterpret_cast<uint32_t*>(&ya);
        uint32_t* ob = reinterpret_cast<uint32_t*>(&yb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 2 * j, f = 2 * j + 1;
          oa[j] = pack_bf16x2(a[e] * c[e] - b[e] * s[e], a[f] * c[f] - b[f] * s[f]);
          ob[j] = pack_bf16x2(b[e] * c[e] + a[e] * s[e], b[f] * c[f] + a[f] * s[f]);
        }
      }
      bf16* y;
      if (is_q)
        y = p.q_out + (row * p.Hq + (h - 2 * p.Hkv)) * D;
      else
        y = (is_v ? p.v_cache : p.k_cache) +
            ((page * p.Hkv + (is_v ? h - p.Hkv : h)) * p.page_size + off) * D;
      *reinterpret_cast<uint4*>(y + i0) = ya;
      *reinterpret_cast<uint4*>(y + i0 + D / 2) = yb;
    }
  }
}

}  // namespace dflash
