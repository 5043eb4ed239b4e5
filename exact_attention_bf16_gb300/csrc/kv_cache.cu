// The paged KV cache's own two operators: planning a step's pages and slots
// from the requests' lengths (attn_kv_plan) and writing its K and V rows
// (attn_kv_append).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
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
// Bound by latency: a few KB to a few hundred KB of slots. Every CTA computes the
// sums itself (the lengths are a few KB in L2) into its shared memory and then
// takes its share of tokens and pages, finding the request of each by bisection.
// Nothing a CTA reads is written except places no other reads (table entries from
// have on, stack entries from c on) and, in place, the lengths and the stack's
// height: then the grid is one cluster, whose barrier stands before those.
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
constexpr int kPlanCtas = 148;  // the most that share a step
static_assert(kMost + 4ll * 1024 * kPlanCtas <= 0xffffffffll, "32-bit token indices do not wrap");

__global__ void kv_plan_kernel(const KvPlanArgs a) {
  extern __shared__ int s_start[];  // cu[n + 1], grow[n + 1], back[n + 1]
  __shared__ Sums warp_sum[32];
  __shared__ int too_wide;
  const int n = a.num_seqs, tid = static_cast<int>(threadIdx.x), nthr = static_cast<int>(blockDim.x);
  const int lane = tid & 31, warp = tid >> 5, nwarps = nthr >> 5;
  int* s_cu = s_start;
  int* s_grow = s_start + n + 1;
  int* s_back = s_start + 2 * (n + 1);
  if (tid == 0) too_wide = 0;
  const int count = max(0, min(*a.free_count, a.free_capacity));
  __syncthreads();
  auto pages = [&](long long tokens) -> long long { return (tokens + a.page_size - 1) >> a.page_shift; };
  // request s: its tokens, pages to take and pages to return
  bool wide = false;
  auto load = [&](int s) -> Sums {
    const int old = max(0, a.seqlens_old[s]), add = a.seqlens_new[s];
    const long long have = pages(old), want = add < 0 ? have : pages(static_cast<long long>(old) + add);
    wide = wide || want > a.max_pages || (add > 0 && static_cast<long long>(old) + add > kMost);
    return Sums{add < 0 ? 0 : add, want - have, add < 0 ? have : 0};
  };
  // every thread sums a run of requests, the runs are scanned by warp and over the warps
  const int run_len = (n + nthr - 1) / nthr, s_begin = min(n, tid * run_len), s_end = min(n, s_begin + run_len);
  Sums mine{0, 0, 0};
#pragma unroll 4
  for (int s = s_begin; s < s_end; ++s) mine = mine + load(s);
  if (wide) too_wide = 1;
  Sums inc = mine;
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
  const Sums total = warp_sum[nwarps - 1];
  Sums at = warp > 0 ? warp_sum[warp - 1] : Sums{0, 0, 0};
  at = Sums{at.add + inc.add - mine.add, at.grow + inc.grow - mine.grow, at.back + inc.back - mine.back};
#pragma unroll 4
  for (int s = s_begin; s < s_end; ++s) {
    s_cu[s] = static_cast<int>(min(at.add, kMost));  // used only where the totals fit (status 0)
    s_grow[s] = static_cast<int>(min(at.grow, kMost));
    s_back[s] = static_cast<int>(min(at.back, kMost));
    at = at + (run_len == 1 ? mine : load(s));
  }
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
  const int rank = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  const int all = nthr * ctas, me = rank * nthr + tid;
  if (status == 0) {
    auto stack = [&](int i) -> int {
      if (i < count) return a.free_pages[i];
      const int e = owner(s_back, n, i - count);
      return a.block_table[e * a.block_table_stride + (i - count - s_back[e])];
    };
    for (uint32_t j = me; j < static_cast<uint32_t>(grow); j += all) {  // (unsigned: as the tokens below)
      const int i = static_cast<int>(j);
      const int s = owner(s_grow, n, i);
      const long long have = pages(max(0, a.seqlens_old[s]));
      a.block_table[s * a.block_table_stride + have + (i - s_grow[s])] = stack(height - 1 - i);
    }
    // ended requests' pages that stay on the stack: a warp copies a row, in order
    if (total.back > 0) {
      for (int s = rank * nwarps + warp; s < n; s += nwarps * ctas) {
        const int len = s_back[s + 1] - s_back[s], keep = min(len, height - grow - count - s_back[s]);
        const int* row = a.block_table + s * a.block_table_stride;
        int* dst = a.free_pages + count + s_back[s];
        for (int i0 = lane; i0 < keep; i0 += 32 * 8) {  // eight loads in flight
          int x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) x[u] = i0 + 32 * u < keep ? row[i0 + 32 * u] : 0;
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (i0 + 32 * u < keep) dst[i0 + 32 * u] = x[u];
        }
      }
    }
    const int tokens = static_cast<int>(total.add);
    // four tokens in a row per thread where there are more tokens than threads: the request and the page are
    // looked up again only where they change
    // (unsigned: the count is below 2^31, and a step past it, at most 4 x 1024 x kPlanCtas, stays below 2^32)
    const uint32_t max_tokens = static_cast<uint32_t>(a.max_tokens);
    const uint32_t run = max_tokens <= static_cast<uint32_t>(all) ? 1 : 4;
    for (uint32_t first = run * me; first < max_tokens; first += run * all) {
      const int t0 = static_cast<int>(first), t1 = static_cast<int>(min(first + run, max_tokens));
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
        if (a.positions != nullptr) a.positions[t] = t < tokens ? pos : -1;
      }
    }
  } else {
    for (uint32_t t = me; t < static_cast<uint32_t>(a.max_tokens); t += all) {
      a.slot_mapping[t] = -1;
      if (a.positions != nullptr) a.positions[t] = -1;
    }
  }
  // every read of the lengths and the stack's height is done (where they are updated in place, the grid is one cluster)
  cg::this_cluster().sync();
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
// tokens, latency-bound for a decode step. The tokens' K and V rows are cut into
// 16-byte units, laid end to end; a block takes 256 kUnits in a row, each thread
// kUnits of them 256 apart, so that eight slots, then eight units, are in flight per
// thread whatever the size of a row, and neighbouring threads read and write
// neighbouring units. Up to one wave of single units takes one per thread (64 tokens
// of 8 x 128: 2.0 us against 2.9).
constexpr int kAppendThreads = 256;

template <int DQK, int DV, int kUnits>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const KvAppendArgs a) {
  constexpr int UK = DQK / 8, UV = DV / 8;  // units of a head's row
  const uint32_t k_units = a.heads_kv * UK, units = k_units + a.heads_kv * UV;  // of a token
  const int64_t slots = static_cast<int64_t>(a.num_pages) << a.page_shift;
  const int64_t total = static_cast<int64_t>(a.tokens) * units;
  constexpr int kBlock = kUnits * kAppendThreads;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kBlock; first < total;
       first += static_cast<int64_t>(gridDim.x) * kBlock) {
    const int64_t t0 = first / units;
    const uint32_t r0 = static_cast<uint32_t>(first - t0 * units) + threadIdx.x;
    int64_t slot[kUnits];
    uint32_t at[kUnits];  // unit of the token
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const uint32_t r = r0 + u * kAppendThreads, t = r / units;
      at[u] = r - t * units;
      slot[u] = first + threadIdx.x + u * kAppendThreads < total ? __ldg(a.slot_mapping + t0 + t) : -1;
    }
    uint4 x[kUnits];
    __nv_bfloat16* dst[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t t = t0 + (r0 + u * kAppendThreads) / units;
      const int64_t page = slot[u] >> a.page_shift, row = slot[u] & (a.page_size - 1);
      const bool is_k = at[u] < k_units;
      const uint32_t v = is_k ? at[u] : at[u] - k_units;
      const uint32_t h = is_k ? v / UK : v / UV, c = 8 * (is_k ? v % UK : v % UV);
      dst[u] = nullptr;
      x[u] = make_uint4(0, 0, 0, 0);
      if (slot[u] >= 0 && slot[u] < slots) {
        dst[u] = is_k ? a.k_cache + page * a.kc_page + row * a.kc_row + h * a.kc_head + c
                      : a.v_cache + page * a.vc_page + row * a.vc_row + h * a.vc_head + c;
        x[u] = __ldcs(reinterpret_cast<const uint4*>(is_k ? a.k + t * a.k_row + h * a.k_head + c
                                                          : a.v + t * a.v_row + h * a.v_head + c));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (dst[u] != nullptr) *reinterpret_cast<uint4*>(dst[u]) = x[u];
  }
}

template <int DQK, int DV>
cudaError_t launch_append(const KvAppendArgs& a, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.tokens) * a.heads_kv * ((DQK + DV) / 8);
  constexpr int64_t kWave = 152 * 8;  // blocks
  const int64_t one = (units + kAppendThreads - 1) / kAppendThreads;
  if (one <= kWave) {
    kv_append_kernel<DQK, DV, 1><<<static_cast<unsigned>(one), kAppendThreads, 0, stream>>>(a);
  } else {
    const int64_t want = (units + 8 * kAppendThreads - 1) / (8 * kAppendThreads);
    kv_append_kernel<DQK, DV, 8><<<static_cast<unsigned>(want < 2 * kWave ? want : 2 * kWave), kAppendThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace kv

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  const int smem = 3 * (a.num_seqs + 1) * static_cast<int>(sizeof(int));
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    cudaError_t r = cudaFuncSetAttribute(kv::kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         3 * (kMaxPlanSeqs + 1) * static_cast<int>(sizeof(int)));
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(kv::kv_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  // A small step is one CTA's work (1000 requests of one token each: 6.4 us). More tokens are shared by up to kPlanCtas
  // (1000 requests with 48,420 tokens 8.3 us, 11.6 by half as many; 3000 with 150,394 tokens 8.3, 11.2 by 64), or where
  // lengths or the stack's height are updated in place, and so must have been read by all first, by a cluster of sixteen,
  // the most there are (12.3 us of the former; eight take 17.1).
  const bool small = a.max_tokens <= 4096 && a.num_seqs <= 1024;
  const bool in_place = a.seqlens_k == a.seqlens_old || a.free_count_out == a.free_count;
  const int shares = static_cast<int>(std::min<int64_t>(kv::kPlanCtas, (static_cast<int64_t>(a.max_tokens) + 1023) / 1024));
  const int ctas = small ? 1 : in_place ? 16 : std::max(16, shares);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(small && a.num_seqs <= 256 && a.max_tokens <= 1024 ? 256 : 1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ctas <= 16 && (small || in_place) ? ctas : 1;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv::kv_plan_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_append(int d_qk, int d_v, const KvAppendArgs& a, cudaStream_t stream) {
  if (d_qk == 64 && d_v == 64) return kv::launch_append<64, 64>(a, stream);
  if (d_qk == 128 && d_v == 128) return kv::launch_append<128, 128>(a, stream);
  if (d_qk == 192 && d_v == 128) return kv::launch_append<192, 128>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace gb300
