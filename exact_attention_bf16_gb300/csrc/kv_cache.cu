// The paged KV cache's own two operators: planning a step's pages and slots
// from the requests' lengths (attn_kv_plan) and writing its K and V rows
// (attn_kv_append).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"

namespace gb300 {
namespace kv {

namespace cg = cooperative_groups;

// ===========================================================================
// Plan
// ===========================================================================
// With add_s = max(new_s, 0), have_s = ceil(old_s / P), want_s = ceil((old_s +
// add_s) / P), grow_s = want_s - have_s (0 when ended) and back_s = have_s when
// ended (else 0), everything follows from the exclusive sums of add, grow and
// back over the requests: the i-th page taken is stack[c + sum(back) - 1 - i],
// where stack is free_pages[0 .. c) followed by the ended requests' pages in
// order, and token t belongs to the request s with cu_s <= t < cu_{s+1}.
//
// Bound by latency: a few KB to a few hundred KB of slots. Every CTA of one
// cluster computes the sums itself (the lengths are a few KB in L2) into its
// shared memory and then takes its share of tokens and pages, finding the
// request of each by bisection. Nothing a CTA reads is written before the
// cluster's barrier except places no other reads (table entries from have on,
// stack entries from c on), so the in-place outputs (lengths, stack height)
// are written after it.
struct Sums {
  long long add, grow, back;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.add + b.add, a.grow + b.grow, a.back + b.back};
}

__device__ __forceinline__ Sums shfl_up(const Sums& v, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, v.add, d), __shfl_up_sync(0xffffffffu, v.grow, d),
              __shfl_up_sync(0xffffffffu, v.back, d)};
}

// Largest s in [0, n) with start[s] <= x, given start[0] <= x < start[n]: the
// one whose range holds x (requests with empty ranges share their start with
// the next and lie before it).
__device__ __forceinline__ int owner(const int* start, int n, int x) {
  int lo = 0, hi = n;  // start[lo] <= x < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

constexpr long long kMost = 0x7fffffff;

__global__ void kv_plan_kernel(const KvPlanArgs a) {
  extern __shared__ int s_start[];  // cu[n + 1], grow[n + 1], back[n + 1]
  __shared__ Sums warp_sum[32];
  __shared__ Sums carry;
  __shared__ int too_wide;
  cg::cluster_group cluster = cg::this_cluster();
  const int n = a.num_seqs, tid = static_cast<int>(threadIdx.x), nthr = static_cast<int>(blockDim.x);
  const int lane = tid & 31, warp = tid >> 5, nwarps = nthr >> 5;
  int* s_cu = s_start;
  int* s_grow = s_start + n + 1;
  int* s_back = s_start + 2 * (n + 1);
  if (tid == 0) {
    carry = Sums{0, 0, 0};
    too_wide = 0;
  }
  const int count = max(0, min(*a.free_count, a.free_capacity));
  __syncthreads();
  auto pages = [&](long long tokens) -> long long { return (tokens + a.page_size - 1) >> a.page_shift; };
  for (int s0 = 0; s0 < n; s0 += nthr) {
    const int s = s0 + tid;
    Sums v{0, 0, 0};
    if (s < n) {
      const int old = max(0, a.seqlens_old[s]), add = a.seqlens_new[s];
      const long long have = pages(old), want = add < 0 ? have : pages(static_cast<long long>(old) + add);
      if (want > a.max_pages || (add > 0 && static_cast<long long>(old) + add > kMost)) too_wide = 1;
      v = Sums{add < 0 ? 0 : add, want - have, add < 0 ? have : 0};
    }
    Sums inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums u = shfl_up(inc, d);
      if (lane >= d) inc = inc + u;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      Sums w = lane < nwarps ? warp_sum[lane] : Sums{0, 0, 0};
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Sums u = shfl_up(w, d);
        if (lane >= d) w = w + u;
      }
      if (lane < nwarps) warp_sum[lane] = w;
    }
    __syncthreads();
    Sums ex = carry + (warp > 0 ? warp_sum[warp - 1] : Sums{0, 0, 0});
    ex = Sums{ex.add + inc.add - v.add, ex.grow + inc.grow - v.grow, ex.back + inc.back - v.back};
    if (s < n) {
      s_cu[s] = static_cast<int>(min(ex.add, kMost));  // used only where the totals fit (status 0)
      s_grow[s] = static_cast<int>(min(ex.grow, kMost));
      s_back[s] = static_cast<int>(min(ex.back, kMost));
    }
    __syncthreads();
    if (tid == 0) carry = carry + warp_sum[nwarps - 1];
    __syncthreads();
  }
  const Sums total = carry;
  if (tid == 0) {
    s_cu[n] = static_cast<int>(min(total.add, kMost));
    s_grow[n] = static_cast<int>(min(total.grow, kMost));
    s_back[n] = static_cast<int>(min(total.back, kMost));
  }
  __syncthreads();
  int status = 0;
  if (total.grow > count + total.back) status = 1;
  else if (too_wide) status = 2;
  else if (total.add > a.max_tokens) status = 3;
  else if (count + total.back > kMost || count + total.back - total.grow > a.free_capacity) status = 4;
  const int height = count + static_cast<int>(min(total.back, kMost - count));  // of the stack, ended pages pushed
  const int grow = static_cast<int>(min(total.grow, kMost));
  const int rank = static_cast<int>(cluster.block_rank());
  const int all = nthr * static_cast<int>(cluster.num_blocks()), me = rank * nthr + tid;
  if (status == 0) {
    auto stack = [&](int i) -> int {
      if (i < count) return a.free_pages[i];
      const int e = owner(s_back, n, i - count);
      return a.block_table[e * a.block_table_stride + (i - count - s_back[e])];
    };
    for (int i = me; i < grow; i += all) {
      const int s = owner(s_grow, n, i);
      const long long have = pages(max(0, a.seqlens_old[s]));
      a.block_table[s * a.block_table_stride + have + (i - s_grow[s])] = stack(height - 1 - i);
    }
    for (int i = count + me; i < height - grow; i += all) a.free_pages[i] = stack(i);
    const int tokens = static_cast<int>(total.add);
    // four tokens in a row per thread where there are more tokens than threads: the request and the page are
    // looked up again only where they change
    const int run = a.max_tokens <= all ? 1 : 4;
    for (int t0 = run * me; t0 < a.max_tokens; t0 += run * all) {
      const int t1 = min(t0 + run, a.max_tokens);
      long long slot = -1;
      int left = 0, end = t0;  // tokens left on the page; first token of the next request
      int s = 0, pos = 0;
      for (int t = t0; t < t1; ++t) {
        if (t >= tokens) {
          slot = -1;
        } else if (left > 0 && t < end) {
          ++slot, --left, ++pos;
        } else {
          if (t >= end || t == t0) {
            s = owner(s_cu, n, t);
            pos = max(0, a.seqlens_old[s]) + (t - s_cu[s]);
            end = s_cu[s + 1];
          } else {
            ++pos;
          }
          const int have = static_cast<int>(pages(max(0, a.seqlens_old[s]))), pi = pos >> a.page_shift;
          const int page = pi < have ? a.block_table[s * a.block_table_stride + pi]
                                     : stack(height - 1 - (s_grow[s] + pi - have));
          slot = (static_cast<long long>(page) << a.page_shift) + (pos & (a.page_size - 1));
          left = a.page_size - 1 - (pos & (a.page_size - 1));
        }
        a.slot_mapping[t] = slot;
      }
    }
  } else {
    for (int t = me; t < a.max_tokens; t += all) a.slot_mapping[t] = -1;
  }
  // every read of the lengths, the stack's height and the old entries is done
  cluster.sync();
  for (int s = me; s <= n; s += all) {
    a.cu_seqlens_q[s] = status == 0 ? s_cu[s] : 0;
    if (s < n) {
      const int old = max(0, a.seqlens_old[s]), add = a.seqlens_new[s];
      a.seqlens_k[s] = status != 0 ? old : (add < 0 ? 0 : old + add);
    }
  }
  if (me == 0) {
    *a.free_count_out = status == 0 ? height - grow : count;
    *a.status = status;
  }
}

// ===========================================================================
// Append
// ===========================================================================
// A pure copy: 2 bytes read and written per element, HBM-bound for a prompt's
// tokens, latency-bound for a decode step. One warp per (token, K or V): its
// heads x d values are 16-byte units, lane after lane, so a row whose heads lie
// side by side is read and written in whole 512-byte runs, eight loads in
// flight per lane before the first store.
template <int D>
__device__ __forceinline__ void append_row(const __nv_bfloat16* src, int64_t src_head, __nv_bfloat16* dst,
                                           int64_t dst_head, int heads, int lane) {
  constexpr int UPH = D / 8, N = 8;
  const int units = heads * UPH;
  for (int i0 = lane; i0 < units; i0 += 32 * N) {
    uint4 x[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = i0 + 32 * u;
      if (i < units) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + (i / UPH) * src_head + 8 * (i % UPH)));
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = i0 + 32 * u;
      if (i < units) *reinterpret_cast<uint4*>(dst + (i / UPH) * dst_head + 8 * (i % UPH)) = x[u];
    }
  }
}

template <int DQK, int DV>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendArgs a) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int64_t slots = static_cast<int64_t>(a.num_pages) << a.page_shift;
  for (int64_t w = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) >> 5; w < 2 * static_cast<int64_t>(a.tokens);
       w += warps) {
    const int64_t t = w >> 1;
    const int64_t slot = a.slot_mapping[t];
    if (slot < 0 || slot >= slots) continue;
    const int64_t page = slot >> a.page_shift, row = slot & (a.page_size - 1);
    if ((w & 1) == 0)
      append_row<DQK>(a.k + t * a.k_row, a.k_head, a.k_cache + page * a.kc_page + row * a.kc_row, a.kc_head, a.heads_kv,
                      lane);
    else
      append_row<DV>(a.v + t * a.v_row, a.v_head, a.v_cache + page * a.vc_page + row * a.vc_row, a.vc_head, a.heads_kv,
                     lane);
  }
}

}  // namespace kv

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  const int smem = 3 * (a.num_seqs + 1) * static_cast<int>(sizeof(int));
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(kv::kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                3 * (kMaxPlanSeqs + 1) * static_cast<int>(sizeof(int)));
  });
  if (e != cudaSuccess) return e;
  // a small step is one CTA's work; more tokens are shared by a cluster of eight
  const bool small = a.max_tokens <= 4096;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(small ? 1 : 8);
  cfg.blockDim = dim3(small && a.num_seqs <= 256 && a.max_tokens <= 1024 ? 256 : 1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cfg.gridDim.x;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv::kv_plan_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_append(int d_qk, int d_v, const KvAppendArgs& a, cudaStream_t stream) {
  const int64_t want = (2 * static_cast<int64_t>(a.tokens) + 7) / 8;  // 8 warps per block
  const unsigned blocks = static_cast<unsigned>(want < 152 * 8 ? want : 152 * 8);
  if (d_qk == 64 && d_v == 64) kv::kv_append_kernel<64, 64><<<blocks, 256, 0, stream>>>(a);
  else if (d_qk == 128 && d_v == 128) kv::kv_append_kernel<128, 128><<<blocks, 256, 0, stream>>>(a);
  else if (d_qk == 192 && d_v == 128) kv::kv_append_kernel<192, 128><<<blocks, 256, 0, stream>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace gb300
