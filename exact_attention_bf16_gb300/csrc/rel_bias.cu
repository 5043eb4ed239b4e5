// The relative position bias laid out by place for the attention kernels
// (rel_bias.cuh), and the sum of its gradient's parts.
#include <cuda_bf16.h>

#include <algorithm>

#include "kernels.h"

namespace gb300 {
namespace rel {

constexpr int kThreads = 256;

__device__ __forceinline__ int bucket_of(const RelTable& t, int r) {
  const int dist = t.two_sided ? abs(r) : max(-r, 0);
  int lo = 0, hi = t.side;  // start[lo] <= dist < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= dist) lo = mid;
    else hi = mid;
  }
  return lo + (t.two_sided && r > 0 ? t.side : 0);
}

// Block (x, y): places of block x, heads of block y; and the buckets of the places, the buckets' ranges, and zeros in the
// gradient's parts, which not every CTA of a packed backward writes. A few hundred KB at most: bound by its launch.
__global__ void __launch_bounds__(kThreads) layout_kernel(const __grid_constant__ RelTable t, float* by_place, uint8_t* bucket,
                                                          int2* range, float4* zero, int64_t n_zero) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int width = 2 * t.reach + 2 * kRelPad;
  const int x = static_cast<int>(blockIdx.x * kThreads + threadIdx.x);
  if (x < width) {
    const int b = bucket_of(t, x - t.reach - kRelPad);
    for (int h = static_cast<int>(blockIdx.y); h < t.heads; h += static_cast<int>(gridDim.y)) {
      const int64_t at = static_cast<int64_t>(b) * t.heads + h;
      const float v = t.f32 ? __ldg(static_cast<const float*>(t.table) + at)
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(t.table)[at]);
      by_place[static_cast<int64_t>(h) * width + x] = v * t.inv_scale;
    }
    if (blockIdx.y == 0) bucket[x] = static_cast<uint8_t>(b);
  }
  if (range != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && static_cast<int>(threadIdx.x) < t.buckets) {
    constexpr int kFar = 0x40000000;
    const int b = static_cast<int>(threadIdx.x), k = b % t.side;
    const int from = t.start[k], to = k + 1 < t.side ? t.start[k + 1] - 1 : kFar;  // distances
    if (b >= t.side) range[b] = make_int2(max(from, 1), to);
    else range[b] = make_int2(-to, k > 0 || t.two_sided ? -from : kFar);
  }
  const int64_t me = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  for (int64_t i = me; i < n_zero; i += static_cast<int64_t>(gridDim.x) * gridDim.y * kThreads)
    zero[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Table entry (bucket, head) = the sum of the head's parts, [rows][buckets]: a block per head, its threads' rows a stride
// apart, then the threads' sums pair by pair.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* parts, int64_t rows, int buckets, int heads, void* out,
                                                         int f32) {
  __shared__ float s[1024];
  const int h = static_cast<int>(blockIdx.x), lanes = static_cast<int>(blockDim.x) / buckets;
  const int b = static_cast<int>(threadIdx.x) % buckets, y = static_cast<int>(threadIdx.x) / buckets;
  float sum = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched before the parts' kernel is over
  if (y < lanes) {
    const float* p = parts + (static_cast<int64_t>(h) * rows) * buckets + b;
#pragma unroll 8
    for (int64_t r = y; r < rows; r += lanes) sum += __ldg(p + r * buckets);
  }
  s[threadIdx.x] = sum;
  __syncthreads();
  for (int n = lanes; n > 1; n = (n + 1) / 2) {  // the upper half onto the lower one
    if (y < n / 2) s[threadIdx.x] += s[(y + (n + 1) / 2) * buckets + b];
    __syncthreads();
  }
  if (y == 0) {
    sum = s[b];
    const int64_t at = static_cast<int64_t>(b) * heads + h;
    if (f32) static_cast<float*>(out)[at] = sum;
    else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(sum);
  }
}

}  // namespace rel

cudaError_t launch_rel_layout(const RelTable& t, const RelBias& b, float* zero, int64_t n_zero, cudaStream_t stream) {
  const int width = 2 * t.reach + 2 * kRelPad;
  const unsigned gx = static_cast<unsigned>((width + rel::kThreads - 1) / rel::kThreads);
  // (rows of blocks beyond the heads only clear: a packed backward of thousands of sequences has tens of MB of parts)
  const int64_t clear = std::min<int64_t>(n_zero / (4 * rel::kThreads), 152 * 8) / gx;
  const unsigned gy = static_cast<unsigned>(std::min<int64_t>(std::max<int64_t>(t.heads, clear), 65535));
  rel::layout_kernel<<<dim3(gx, gy), rel::kThreads, 0, stream>>>(t, const_cast<float*>(b.by_place), const_cast<uint8_t*>(b.bucket),
                                                                 const_cast<int2*>(b.range), reinterpret_cast<float4*>(zero),
                                                                 n_zero / 4);
  return cudaGetLastError();
}

cudaError_t launch_rel_sum(const float* parts, int64_t rows, int buckets, int heads, void* out, int f32, cudaStream_t stream) {
  return launch_early(rel::sum_parts_kernel, dim3(static_cast<unsigned>(heads)), 1024, 0, stream, parts, rows, buckets, heads, out,
                      f32);
}

}  // namespace gb300
