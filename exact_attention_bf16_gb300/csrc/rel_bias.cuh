// Learned relative position bias by buckets, as the kernels read it. The bias of
// a (query, key) pair depends on the head and on r = key - query's position
// alone, and beyond a reach R on r's sign alone: the bucket borders lie within
// |r| <= R. A call first lays it out by r (rel_layout.cuh): one row of fp32 per
// head, over the softmax scale (in units of the raw logits q . k), of
// r = -R - kRelPad .. R + kRelPad - 1. A tile of logits that lies beyond the reach
// as a whole then takes one number, added to the softmax's own offset; any other
// takes one load per logit, neighbouring lanes neighbouring addresses, from a
// row wide enough that no index needs a test.
//
// What it costs: at N = 8192 (B2, 16 heads over 4, d = 128, causal, 32 buckets up to 128) the forward 387 us against
// 367 without a bias and the backward 1444 against 1396; at N = 512 (B32, 16 heads, d = 64, both sides, half of the warps'
// tiles within the reach) 89 against 84 and 327 against 283, 27 of them for the table's gradient.
#pragma once
#include "kernels.h"
#include "ptx_sm100.cuh"

namespace gb300 {

// A head's row: in shared memory from r = -reach - PAD on (SMEM: kernels that keep it there where it fits, b.in_smem; smem is its
// address), or in L1. Nothing of it lives in registers between tiles.
template <int PAD, bool SMEM = true>
struct RelRow {
  const RelBias& b;
  uint32_t smem;
  int h;
  __device__ __forceinline__ bool in_smem() const { return SMEM && b.in_smem; }
  __device__ __forceinline__ const float* global() const {  // of r = 0
    return b.by_place + static_cast<int64_t>(h) * (2 * b.reach + 2 * kRelPad) + b.reach + kRelPad;
  }
  __device__ __forceinline__ uint32_t shared() const { return smem + 4 * (b.reach + PAD); }
  // Copied by n threads, which then have to meet.
  __device__ __forceinline__ void load(int thread, int n) const {
    const float* src = global() - b.reach - PAD;
    for (int x = thread; x < 2 * (b.reach + PAD); x += n) st_shared_f32(smem + 4 * x, __ldg(src + x));
  }
  __device__ __forceinline__ float one(int r) const { return in_smem() ? ld_shared_f32(shared() + 4 * r) : __ldg(global() + r); }
  // Whether places r_min .. r_max all have one bias, `add`.
  __device__ __forceinline__ bool far(int r_min, int r_max, float& add) const {
    const bool l = r_max <= -b.reach, r = r_min >= b.reach;
    add = 0.f;
    if (l || r) add = one(l ? -b.reach : b.reach);
    return l || r;
  }
  // The same with the two numbers in registers (left of and right of the reach).
  __device__ __forceinline__ float2 both() const { return make_float2(one(-b.reach), one(b.reach)); }
  __device__ __forceinline__ bool far(int r_min, int r_max, const float2& lr, float& add) const {
    const bool l = r_max <= -b.reach, r = r_min >= b.reach;
    add = l ? lr.x : r ? lr.y : 0.f;
    return l || r;
  }
  // The buckets of its places lie behind the row in shared memory, if they are asked for.
  static constexpr int bytes(int reach) { return 5 * 2 * (reach + PAD); }
  __device__ __forceinline__ void load_buckets(int thread, int n) const {
    const int width = 2 * (b.reach + PAD);
    for (int x = thread; x < width; x += n) st_shared_u8(smem + 4 * width + x, __ldg(b.bucket + kRelPad - PAD + x));
  }
  __device__ __forceinline__ int bucket(int r) const {
    return in_smem() ? ld_shared_u8(smem + 4 * 2 * (b.reach + PAD) + b.reach + PAD + r) : __ldg(b.bucket + kRelPad + b.reach + r);
  }
  // Whether places r_min .. r_max all lie beyond the reach or (id: it, else -1) in one bucket within it.
  __device__ __forceinline__ bool far_or_one(int r_min, int r_max, float& add, int& id) const {
    id = -1;
    if (far(r_min, r_max, add)) return true;
    if (r_min < -b.reach || r_max > b.reach) return false;  // in two
    id = bucket(r_min);
    if (id != bucket(r_max)) id = -1;
    if (id >= 0) add = one(r_min);
    return id >= 0;
  }
  // f(load) with load(c) the bias of place r + c.
  template <typename F>
  __device__ __forceinline__ void at(int r, F&& f) const {
    if (in_smem()) {
      const uint32_t from = shared() + 4 * r;
      f([from](int c) { return ld_shared_f32(from + 4 * c); });
    } else {
      const float* from = global() + r;
      f([from](int c) { return __ldg(from + c); });
    }
  }
};

// A head's row in L1 as paged_kernel reads it: by itself, or (FOURS, three or more heads that share a K/V head) place by place
// among four of them (RelTable::fours): a warp's rows are a few tokens of all these heads, and a load takes a step per line. Chunks of
// 300 to 1500 tokens over up to 8192 keys, by themselves and in fours: 12 heads over 4 99 and 98 us, 16 over 4 120 and 114, 15 over 3 112
// and 111, 12 over 2 93 and 92, 14 over 2 89 and 87, 16 over 2 112 and 109, 16 over 1 110 and 100. Two heads leave half of every line
// empty: 16 over 8 123 and 135. (All heads of the group side by side, a stride known at run time: 126 for 127 of 16 over 4, but 16 over
// 16 156 for 148.) Not where one tile of rows holds any request's tokens (16 requests of 20: 56.3 us so, 55.0).
template <bool FOURS>
struct RelPaged {
  const RelBias& b;
  const float* at0;  // of place 0
  bool fours;
  __device__ __forceinline__ RelPaged(const RelBias& bias, int hk, int group, int h) : b(bias), fours(FOURS && rel_in_fours(group)) {
    const int64_t width = 2 * bias.reach + 2 * kRelPad, zero = bias.reach + kRelPad;
    at0 = fours ? bias.by_place + 4 * ((static_cast<int64_t>(hk) * ((group + 3) / 4) + h / 4) * width + zero) + h % 4
                : bias.by_place + (static_cast<int64_t>(hk) * group + h) * width + zero;
  }
  __device__ __forceinline__ bool far(int r_min, int r_max, float& add) const {
    const bool l = r_max <= -b.reach, r = r_min >= b.reach;
    const int at = l ? -b.reach : b.reach;
    add = l || r ? __ldg(at0 + (fours ? 4 * at : at)) : 0.f;
    return l || r;
  }
  // f(load) with load(c) the bias of place r + c.
  template <typename F>
  __device__ __forceinline__ void at(int r, F&& f) const {
    if (fours) {
      const float* from = at0 + 4 * r;
      f([from](int c) { return __ldg(from + 4 * c); });
    } else {
      const float* from = at0 + r;
      f([from](int c) { return __ldg(from + c); });
    }
  }
};

// What the dQ kernel holds of the gradient in shared memory: each warp's sums by bucket, the halves' sums of a row, and behind
// them, where the row is there too (b.in_smem), the buckets' first and last places, the row and its places' buckets.
constexpr int kRelRowSums = 2 * 128 * 4, kRelSums = 8 * kRelMaxBuckets * 4 + kRelRowSums, kRelRange = kRelMaxBuckets * 8;  // bytes
template <int PAD>
struct RelGrad {
  const RelBias& b;
  uint32_t smem;
  static constexpr int bytes(int reach) { return kRelSums + kRelRange + 5 * 2 * (reach + PAD); }  // with the row
  __device__ __forceinline__ uint32_t row() const { return smem + kRelSums + kRelRange; }
  __device__ __forceinline__ uint32_t row_sum(int half, int row) const { return smem + kRelSums - kRelRowSums + 4 * (128 * half + row); }
  __device__ __forceinline__ uint32_t sum(int warp, int bucket) const { return smem + 4 * (warp * kRelMaxBuckets + bucket); }
  // Brings what load() and RelRow::load() read into L1 (their latency was a third of a microsecond of every CTA).
  __device__ __forceinline__ void prefetch(const float* row, int thread, int n) const {
    if (!b.in_smem || b.parts == nullptr) return;
    const int width = 2 * (b.reach + PAD);
    for (int x = 32 * thread; x < width; x += 32 * n) touch_global(row + x);
    for (int x = 128 * thread; x < width; x += 128 * n) touch_global(b.bucket + kRelPad - PAD + x);
    for (int x = 16 * thread; x < b.buckets; x += 16 * n) touch_global(b.range + x);
  }
  // By n threads, which then have to meet.
  __device__ __forceinline__ void load(int thread, int n) const {
    for (int x = thread; x < 8 * kRelMaxBuckets; x += n) st_shared_f32(smem + 4 * x, 0.f);
    if (!b.in_smem || b.parts == nullptr) return;
    const int width = 2 * (b.reach + PAD);
    for (int x = thread; x < b.buckets; x += n) {
      const int2 r = __ldg(b.range + x);
      st_shared_f32(smem + kRelSums + 8 * x, __int_as_float(r.x));
      st_shared_f32(smem + kRelSums + 8 * x + 4, __int_as_float(r.y));
    }
    for (int x = thread; x < width; x += n) st_shared_u8(row() + 4 * width + x, __ldg(b.bucket + kRelPad - PAD + x));
  }
  __device__ __forceinline__ int bucket(int r) const {
    return b.in_smem ? ld_shared_u8(row() + 4 * 2 * (b.reach + PAD) + b.reach + PAD + r) : __ldg(b.bucket + kRelPad + b.reach + r);
  }
  __device__ __forceinline__ int2 range(int bucket) const {
    if (!b.in_smem) return __ldg(b.range + bucket);
    return make_int2(__float_as_int(ld_shared_f32(smem + kRelSums + 8 * bucket)),
                     __float_as_int(ld_shared_f32(smem + kRelSums + 8 * bucket + 4)));
  }
  // Adds the sum of x over the warp to a bucket.
  __device__ __forceinline__ void add(int warp, int bucket, float x) const {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if (bucket % 32 == static_cast<int>(lane_id())) st_shared_f32(sum(warp, bucket), ld_shared_f32(sum(warp, bucket)) + x);
  }
  // Adds the diagonals' sums t of a block (diagonal_sums), whose place at row 0, column 0 is r00. Each window of 32 places is
  // summed by bucket along the lanes (a bucket's places lie side by side), and the lane that bucket lane + 32 k belongs to takes
  // the sum from the last of them.
  __device__ __forceinline__ void add(int warp, const float (&t)[3], int r00) const {
    const int lane = static_cast<int>(lane_id());
    float x[3];
    int start[3];  // first lane of this one's bucket
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int id = bucket(r00 + 32 * q - lane), before = __shfl_up_sync(0xffffffffu, id, 1);
      const uint32_t heads = __ballot_sync(0xffffffffu, lane == 0 || id != before);
      start[q] = 31 - __clz(heads & (0xffffffffu >> (31 - lane)));
      x[q] = t[q];
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const float y = __shfl_up_sync(0xffffffffu, x[q], d);
        if (lane - d >= start[q]) x[q] += y;
      }
    }
    for (int k = 0; 32 * k < b.buckets; ++k) {
      const bool mine = lane + 32 * k < b.buckets;
      const int2 places = mine ? range(lane + 32 * k) : make_int2(1, 0);
      float all = 0.f;
#pragma unroll
      for (int q = 0; q < 3; ++q) {  // places top .. top - 31
        const int top = r00 + 32 * q, low = max(places.x, top - 31);
        const float y = __shfl_sync(0xffffffffu, x[q], (top - low) & 31);
        if (low <= min(places.y, top)) all += y;
      }
      if (mine) st_shared_f32(sum(warp, lane + 32 * k), ld_shared_f32(sum(warp, lane + 32 * k)) + all);
    }
  }
};

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

}  // namespace gb300
