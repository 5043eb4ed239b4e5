// The relative position bias laid out by place for the attention kernels
// (rel_layout.cuh), and the sum of its gradient's parts.
#include <cuda_bf16.h>

#include <algorithm>

#include "kernels.h"
#include "rel_layout.cuh"

namespace gb300 {
namespace rel {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) layout_kernel(const __grid_constant__ RelLayout l) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  rel_layout(l, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
}

// Table entry (bucket, head) = the sum of the head's parts, [rows][buckets]: a block per head, its threads' rows a stride
// apart, then the threads' sums pair by pair.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* parts, int64_t rows, int buckets, int heads, void* out,
                                                         int f32) {
  __shared__ float s[1024];
  const int h = static_cast<int>(blockIdx.x), lanes = static_cast<int>(blockDim.x) / buckets;
  const int b = static_cast<int>(threadIdx.x) % buckets, y = static_cast<int>(threadIdx.x) / buckets;
  float sum = 0.f;
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
  // Beside the dK/dV kernel, behind the parts' kernel: over before this one is. (Behind both, the backward of
  // 7 packed sequences of up to 500 took 39.3 us, 38.1 so; of 32 x 512, 16 heads, 329 and 326.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace rel

int rel_layout_blocks(const RelLayout& l, int threads, int most) {
  const int64_t items = std::max<int64_t>((2 * l.table.reach + 2 * kRelPad) * rel_rows(l.table), l.n_zero);
  return static_cast<int>(std::min<int64_t>((items + threads - 1) / threads, most));
}

cudaError_t launch_rel_layout(const RelLayout& l, cudaStream_t stream) {
  rel::layout_kernel<<<rel_layout_blocks(l, rel::kThreads, 152 * 8), rel::kThreads, 0, stream>>>(l);
  return cudaGetLastError();
}

cudaError_t launch_rel_sum(const float* parts, int64_t rows, int buckets, int heads, void* out, int f32, cudaStream_t stream) {
  return launch_early(rel::sum_parts_kernel, dim3(static_cast<unsigned>(heads)), 1024, 0, stream, parts, rows, buckets, heads, out,
                      f32);
}

}  // namespace gb300
