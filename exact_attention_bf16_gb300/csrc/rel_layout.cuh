// The relative position bias laid out by place (rel_bias.cuh), by blocks of a kernel of its own (rel_bias.cu) or of the
// tile lists' (schedule.cu).
#pragma once
#include <cuda_bf16.h>

#include "kernels.h"

namespace gb300 {

__device__ __forceinline__ int rel_bucket(const RelTable& t, int r) {
  const int dist = t.two_sided ? abs(r) : max(-r, 0);
  int lo = 0, hi = t.side;  // start[lo] <= dist < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= dist) lo = mid;
    else hi = mid;
  }
  return lo + (t.two_sided && r > 0 ? t.side : 0);
}

// Block `block` of `blocks`: its share of (head, place), and of the places' buckets, the buckets' ranges, and zeros in the
// gradient's parts, which not every CTA of a packed backward writes.
__device__ __forceinline__ void rel_layout(const RelLayout& l, int block, int blocks) {
  const RelTable& t = l.table;
  const int width = 2 * t.reach + 2 * kRelPad;
  const int64_t all = static_cast<int64_t>(width) * rel_rows(t), step = static_cast<int64_t>(blocks) * blockDim.x;
  const int64_t me = static_cast<int64_t>(block) * blockDim.x + threadIdx.x;
  for (int64_t i = me; i < all; i += step) {
    const int64_t y = t.fours > 0 ? i >> 2 : i;
    int h = static_cast<int>(y / width);
    const int x = static_cast<int>(y - static_cast<int64_t>(h) * width);
    if (t.fours > 0) {
      const int hk = h / t.fours, g = 4 * (h - hk * t.fours) + static_cast<int>(i & 3);
      if (g >= t.group) continue;
      h = hk * t.group + g;
    }
    const int b = rel_bucket(t, x - t.reach - kRelPad);
    const int64_t at = static_cast<int64_t>(b) * t.heads + h;
    float v = t.f32 ? __ldg(static_cast<const float*>(t.table) + at)
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(t.table)[at]);
    if (isfinite(v)) v = fminf(fmaxf(v, -kRelMaxEntry), kRelMaxEntry);
    l.by_place[i] = v * t.inv_scale;
    if (h == 0) l.bucket[x] = static_cast<uint8_t>(b);
  }
  if (l.range != nullptr && me < t.buckets) {
    constexpr int kFar = 0x40000000;
    const int b = static_cast<int>(me), k = b % t.side;
    const int from = t.start[k], to = k + 1 < t.side ? t.start[k + 1] - 1 : kFar;  // distances
    if (b >= t.side) l.range[b] = make_int2(max(from, 1), to);
    else l.range[b] = make_int2(-to, k > 0 || t.two_sided ? -from : kFar);
  }
  for (int64_t i = me; i < l.n_zero; i += step) l.zero[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (l.zero_word != nullptr && me == 0) *l.zero_word = 0;
}

}  // namespace gb300
