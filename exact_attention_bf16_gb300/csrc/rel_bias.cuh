// Learned relative position bias by buckets, as the kernels read it. The bias of
// a (query, key) pair depends on the head and on r = key - query's position
// alone, and beyond a reach R on r's sign alone: the bucket borders lie within
// |r| <= R. A call first lays it out by r (rel_bias.cu): one row of fp32 per
// head, times log2(e), of r = -R - kRelPad .. R + kRelPad - 1. A tile of logits that lies beyond the reach as a whole then
// takes one number, added for free to the softmax's own offset; any other takes
// one load per logit, neighbouring lanes neighbouring addresses (the row in L1: 3 KB
// at R = 128), from a row wide enough that no index needs a test.
#pragma once
#include "kernels.h"
#include "ptx_sm100.cuh"

namespace gb300 {

// A head's row.
struct RelRow {
  const float* centre;  // centre[r], -reach - kRelPad <= r < reach + kRelPad
  float left, right;    // of r <= -reach and r >= reach
  int reach;
};
__device__ __forceinline__ RelRow rel_row(const RelBias& b, int h) {
  const float* row = b.by_place + static_cast<int64_t>(h) * (2 * b.reach + 2 * kRelPad);
  return RelRow{row + b.reach + kRelPad, __ldg(row + kRelPad), __ldg(row + 2 * b.reach + kRelPad), b.reach};
}
// Whether places r_min .. r_max all have one bias, `add`.
__device__ __forceinline__ bool rel_far(const RelRow& w, int r_min, int r_max, float& add) {
  const bool l = r_max <= -w.reach, r = r_min >= w.reach;
  add = l ? w.left : r ? w.right : 0.f;
  return l || r;
}

// Sums along the diagonals of a warp's 32 x 64 block, lane l's row in x[0 .. 63]: t[q] of lane l becomes
// sum_i x_i[d + i], d = 32 q - l, over the lanes i with 0 <= d + i < 64. Five rounds, in each of which two lanes a power of
// two apart trade half of their numbers and add the rest: entry k of the lanes that differ from l in the bits above the round's
// is the sum along the diagonal 2^round k - (l's bits up to it). 62 shuffles in all, in a fixed order of additions.
__device__ __forceinline__ void diagonal_sums(float (&x)[64], float (&t)[3]) {
  const int lane = static_cast<int>(lane_id());
  auto round = [&](auto n_tag, int bit) {
    constexpr int n = decltype(n_tag)::value;
    const bool odd = (lane & bit) != 0;
    float prev = 0.f;
    float last = 0.f;
#pragma unroll
    for (int j = 0; j <= n / 2; ++j) {
      const float own = 2 * j < n ? x[2 * j] : 0.f;
      const float got = 2 * j + 1 < n ? __shfl_xor_sync(0xffffffffu, x[2 * j + 1], bit) : 0.f;
      const float sum = own + (odd ? prev : got);
      if (j < 64) x[j] = sum;
      last = sum;
      prev = got;
    }
    return last;
  };
  round(std::integral_constant<int, 64>{}, 1);
  round(std::integral_constant<int, 33>{}, 2);
  round(std::integral_constant<int, 17>{}, 4);
  round(std::integral_constant<int, 9>{}, 8);
  round(std::integral_constant<int, 5>{}, 16);
  t[0] = x[0], t[1] = x[1], t[2] = x[2];
}

// Adds the diagonals' sums t of a block (diagonal_sums), whose place at row 0, column 0 is r00, to the buckets' sums: bucket
// lane + 32 k in acc[k]. Each window of 32 places is summed by bucket along the lanes (a bucket's places lie side by side), and
// the bucket's lane takes the sum from the last of them.
__device__ __forceinline__ void bucket_sums(const RelBias& b, const float (&t)[3], int r00, float (&acc)[4]) {
  const int lane = static_cast<int>(lane_id());
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int top = r00 + 32 * q, r = top - lane;  // places top .. top - 31
    const int id = __ldg(b.bucket + r + b.reach + kRelPad);
    const int before = __shfl_up_sync(0xffffffffu, id, 1);
    const uint32_t heads = __ballot_sync(0xffffffffu, lane == 0 || id != before);
    const int start = 31 - __clz(heads & (0xffffffffu >> (31 - lane)));
    float x = t[q];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane - d >= start) x += y;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (32 * k >= b.buckets) break;
      const int2 range = lane + 32 * k < b.buckets ? __ldg(b.range + lane + 32 * k) : make_int2(1, 0);
      const int low = max(range.x, top - 31);
      const float y = __shfl_sync(0xffffffffu, x, (top - low) & 31);
      if (low <= min(range.y, top)) acc[k] += y;
    }
  }
}

}  // namespace gb300
