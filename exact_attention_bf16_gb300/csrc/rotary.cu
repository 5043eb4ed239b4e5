// Rotary position encoding: queries and keys of training batches
// (attn_rotary), and keys on their way into the paged cache with the queries
// beside them (attn_kv_append_rotary).
//
// With a row's position p, pair (x, y) of frequency f becomes
//   (x c - y s, x s + y c),  c = cos[p][f], s = sin[p][f],
// three operations per number against 4 bytes moved: HBM-bound for a prompt's
// tokens, bound by latency for a decode step.
//
// A thread takes 16 columns of a head, the eight pairs of eight neighbouring
// frequencies: two 16-byte units of the row, side by side or half of the rotated
// part apart, and the same 64 bytes of the tables either way. It takes them of kHeads heads, so
// that a table row, which all heads of a token share, is read once for kHeads
// rows of data. The data are loaded before the position is known and the tables
// behind it, so that a small call waits twice, not three times. What is not rotated
// goes along in units of its own, V in blocks of their own behind the others.
//
// 20011 tokens of 32 heads over 8, d = 128, into the cache: 81 us for 502 MB, 6.2 TB/s; 40001 packed tokens and their
// gradients, two calls: 250 us for 1.64 GB, 6.6 TB/s (a copy reaches 6.8). By the heads a thread takes (1, 2, 4, 8) with blocks of
// 256: 105, 88, 97 and 113 us of the former; by the block's threads (64, 128, 256) with two heads: 84, 84 and 88: small blocks
// leave less of an SM waiting for a block's last loads. Stores that L2 lets go first: 256 -> 249 us of the latter. Up to a wave
// of threads one head each: 1000 packed tokens of 16 heads over 4, d = 64, and their gradients 5.6 us, 6.1 with two (100 tokens 4.1
// and 4.5, 2999 tokens 8.5 and 8.8; 64 tokens of 32 heads over 8, d = 192, into the cache 2.7 and 2.6).
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"

namespace gb300 {
namespace rotary {

constexpr int kThreads = 128;
constexpr int kVUnits = 4;  // 16-byte units of V per thread

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t pack(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The eight pairs in x, y: halves (x_e, y_e), or adjacent (x_0, x_1), (x_2, x_3), ... (y_6, y_7).
template <bool ADJ>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
  uint32_t* xw = &x.x;
  uint32_t* yw = &y.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = unpack(xw[e]), b = unpack(yw[e]);
    if constexpr (ADJ) {
      xw[e] = pack(fmaf(a.x, c[e], -a.y * s[e]), fmaf(a.x, s[e], a.y * c[e]));
      yw[e] = pack(fmaf(b.x, c[e + 4], -b.y * s[e + 4]), fmaf(b.x, s[e + 4], b.y * c[e + 4]));
    } else {
      xw[e] = pack(fmaf(a.x, c[2 * e], -b.x * s[2 * e]), fmaf(a.y, c[2 * e + 1], -b.y * s[2 * e + 1]));
      yw[e] = pack(fmaf(a.x, s[2 * e], b.x * c[2 * e]), fmaf(a.y, s[2 * e + 1], b.y * c[2 * e + 1]));
    }
  }
}

__device__ __forceinline__ int position(const RotaryArgs& a, uint32_t b, uint32_t n) {
  return a.positions != nullptr ? __ldg(a.positions + b * a.pos_b + n) : static_cast<int>(n);
}

// Blocks 0 .. rot_blocks - 1: 16 columns of kHeads heads per thread, heads g, g + groups, ... of the q heads and then the
// k heads; the others: V's units, laid end to end.
template <int D, int kHeads, bool ADJ>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, uint32_t groups, uint32_t rot_blocks) {
  const int64_t slots = static_cast<int64_t>(a.num_pages) << a.page_shift;
  if (blockIdx.x >= rot_blocks) {
    const uint32_t per_head = a.d_v / 8, units = a.heads_kv * per_head;
    const uint64_t first = static_cast<uint64_t>(blockIdx.x - rot_blocks) * (kThreads * kVUnits);
    const uint32_t t0 = static_cast<uint32_t>(first / units);
    const uint32_t r0 = static_cast<uint32_t>(first - static_cast<uint64_t>(t0) * units) + threadIdx.x;
    uint4 x[kVUnits];
    __nv_bfloat16* dst[kVUnits];
#pragma unroll
    for (int u = 0; u < kVUnits; ++u) {
      const uint32_t r = r0 + u * kThreads, dt = r / units, at = r - dt * units;
      const uint64_t t = static_cast<uint64_t>(t0) + dt;
      dst[u] = nullptr;
      if (t >= a.tokens) continue;
      const uint32_t h = at / per_head, c = 8 * (at - h * per_head);
      x[u] = __ldcs(reinterpret_cast<const uint4*>(a.v + static_cast<int64_t>(t) * a.v_row + h * a.v_head + c));
      const int64_t slot = __ldg(a.slots + t);
      if (slot >= 0 && slot < slots && static_cast<uint32_t>(position(a, 0, static_cast<uint32_t>(t))) < a.num_positions)
        dst[u] = a.v_out + (slot >> a.page_shift) * a.vo_page + (slot & (a.page_size - 1)) * a.vo_row + h * a.vo_head + c;
    }
#pragma unroll
    for (int u = 0; u < kVUnits; ++u)
      if (dst[u] != nullptr) *reinterpret_cast<uint4*>(dst[u]) = x[u];
    return;
  }
  constexpr uint32_t kItems = D / 16;
  const uint32_t per_token = groups * kItems;
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * kThreads;
  const uint32_t t0 = static_cast<uint32_t>(first / per_token);
  const uint32_t r0 = static_cast<uint32_t>(first - static_cast<uint64_t>(t0) * per_token) + threadIdx.x, dt = r0 / per_token;
  const uint64_t t = static_cast<uint64_t>(t0) + dt;
  if (t >= a.tokens) return;
  const uint32_t r = r0 - dt * per_token, g = r / kItems, i = r - g * kItems;
  uint32_t b = 0, n = static_cast<uint32_t>(t);
  if (a.seqlen != a.tokens) b = n / a.seqlen, n -= b * a.seqlen;
  const uint32_t rotated = a.rot / 16;
  uint32_t c0, c1;  // the two units' columns
  if (i < rotated) {
    c0 = a.first + (ADJ ? 16 * i : 8 * i);
    c1 = c0 + (ADJ ? 8 : a.rot / 2);
  } else {
    c0 = 16 * (i - rotated), c1 = c0 + 8;
    if (c0 >= a.first) c0 += a.rot;
    if (c1 >= a.first) c1 += a.rot;
  }
  uint4 x[kHeads], y[kHeads];
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    const uint32_t h = g + u * groups;
    const __nv_bfloat16* src = nullptr;
    if (h < a.heads) src = a.q + b * a.q_b + n * a.q_row + h * a.q_head;
    else if (h < a.heads + a.heads_kv) src = a.k + b * a.k_b + n * a.k_row + (h - a.heads) * a.k_head;
    if (src != nullptr) {
      x[u] = *reinterpret_cast<const uint4*>(src + c0);
      y[u] = *reinterpret_cast<const uint4*>(src + c1);
    }
  }
  const int64_t slot = a.slots != nullptr ? __ldg(a.slots + t) : 0;
  const uint32_t pos = static_cast<uint32_t>(position(a, b, n));
  if (pos >= a.num_positions) return;
  if (i < rotated) {
    float c[8], s[8];
    const float4* ct = reinterpret_cast<const float4*>(a.cos + pos * a.table_row + 8 * i);
    const float4* st = reinterpret_cast<const float4*>(a.sin + pos * a.table_row + 8 * i);
    const float4 ca = __ldg(ct), cb = __ldg(ct + 1), sa = __ldg(st), sb = __ldg(st + 1);
    c[0] = ca.x, c[1] = ca.y, c[2] = ca.z, c[3] = ca.w, c[4] = cb.x, c[5] = cb.y, c[6] = cb.z, c[7] = cb.w;
    s[0] = sa.x, s[1] = sa.y, s[2] = sa.z, s[3] = sa.w, s[4] = sb.x, s[5] = sb.y, s[6] = sb.z, s[7] = sb.w;
    if (a.inverse) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = -s[e];
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      if (g + u * groups < a.heads + a.heads_kv) turn<ADJ>(x[u], y[u], c, s);
  }
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    const uint32_t h = g + u * groups;
    __nv_bfloat16* dst = nullptr;
    if (h < a.heads) {
      dst = a.q_out + b * a.qo_b + n * a.qo_row + h * a.qo_head;
    } else if (h < a.heads + a.heads_kv) {
      if (a.slots == nullptr) dst = a.k_out + b * a.ko_b + n * a.ko_row + (h - a.heads) * a.ko_head;
      else if (slot >= 0 && slot < slots)
        dst = a.k_out + (slot >> a.page_shift) * a.ko_b + (slot & (a.page_size - 1)) * a.ko_row + (h - a.heads) * a.ko_head;
    }
    if (dst != nullptr) {
      __stcs(reinterpret_cast<uint4*>(dst + c0), x[u]);
      __stcs(reinterpret_cast<uint4*>(dst + c1), y[u]);
    }
  }
}

template <int D, int kHeads>
cudaError_t launch_h(const RotaryArgs& a, cudaStream_t stream) {
  const uint32_t heads = a.heads + a.heads_kv, groups = (heads + kHeads - 1) / kHeads;
  const uint64_t items = static_cast<uint64_t>(a.tokens) * groups * (D / 16);
  const uint64_t v_units = a.v != nullptr ? static_cast<uint64_t>(a.tokens) * a.heads_kv * (a.d_v / 8) : 0;
  const uint64_t rot_blocks = (items + kThreads - 1) / kThreads;
  const uint64_t blocks = rot_blocks + (v_units + kThreads * kVUnits - 1) / (kThreads * kVUnits);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto kern = a.interleaved ? rotary_kernel<D, kHeads, true> : rotary_kernel<D, kHeads, false>;
  kern<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, groups, static_cast<uint32_t>(rot_blocks));
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const RotaryArgs& a, cudaStream_t stream) {
  const uint64_t items = static_cast<uint64_t>(a.tokens) * (a.heads + a.heads_kv) * (D / 16);
  return items <= 152 * 2048 ? launch_h<D, 1>(a, stream) : launch_h<D, 2>(a, stream);
}

}  // namespace rotary

cudaError_t launch_rotary(int d_qk, const RotaryArgs& a, cudaStream_t stream) {
  if (d_qk == 64) return rotary::launch_d<64>(a, stream);
  if (d_qk == 128) return rotary::launch_d<128>(a, stream);
  if (d_qk == 192) return rotary::launch_d<192>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace gb300
