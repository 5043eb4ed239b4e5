// Work lists for packed variable-length batches (the tile scheduler for
// variable-length balance of newton wiki "FlashAttention-4", 核心技術).
//
// A variable-length launch has one CTA per (sequence, head, block of R rows).
// Without a list the grid must be sized for the longest sequence in every
// sequence, and the CTAs past a shorter sequence's end start only to exit;
// the sequences also run in their packed order, so a long sequence packed last
// leaves the GPU half idle at the end. The list built here has exactly one
// entry per real block, ordered so that the sequences with the most blocks
// come first (longest processing time first), then head by head, then the
// blocks of each head heaviest first as the kernels' own order has them, so
// that a head's CTAs still run together and share its K/V in L2. The grid is
// sized by an upper bound the host knows (heads * (total / R + sequences));
// entries past the real count are empty and their CTAs exit at once.
//
// One block builds the list: a counting sort of the sequences by block count
// (bins in shared memory), a scan over the bins from the largest count down,
// then one warp per sequence writes its entries. Sequences with the same
// block count are placed in arrival order of an atomic counter; the order
// affects only scheduling, never a result.
//
// The same launch makes the sequences' tensor maps (SeqMaps), a warp per map.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "kernels.h"
#include "ptx_sm100.cuh"

namespace gb300 {
namespace sched {

constexpr int kThreads = 1024;
constexpr int kSharedSeqs = 1024;  // up to so many sequences need no scratch in global memory

// Block b < n_lists builds list b (a backward's two lists in one launch), the blocks behind them the tensor maps.
__global__ void __launch_bounds__(kThreads, 1)
    tile_list_kernel(const int* cu_q, const int* cu_k, int num_seqs, TileListSpec l0, TileListSpec l1, int n_lists,
                     int64_t* scratch, uint32_t* zero_word, const __grid_constant__ SeqMaps maps) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next kernel reads no list and no map
  if (static_cast<int>(blockIdx.x) >= n_lists) {
    __shared__ alignas(128) uint32_t s_map[kThreads / 32][32];
    const int ln = static_cast<int>(threadIdx.x & 31u), wp = static_cast<int>(threadIdx.x >> 5);
    const int64_t count = static_cast<int64_t>(num_seqs) * maps.n;
    for (int64_t x = (static_cast<int64_t>(blockIdx.x) - n_lists) * (kThreads / 32) + wp; x < count;
         x += (static_cast<int64_t>(gridDim.x) - n_lists) * (kThreads / 32)) {
      const int s = static_cast<int>(x / maps.n), m = static_cast<int>(x - static_cast<int64_t>(s) * maps.n);
      s_map[wp][ln] = reinterpret_cast<const uint32_t*>(&maps.base[m])[ln];
      __syncwarp();
      if (ln == 0) {
        const int end = maps.by_keys[m] ? min(cu_k[s + 1], maps.rows_k) : min(cu_q[s + 1], maps.rows_q);
        tensormap_set_dim2(s_map[wp], static_cast<uint32_t>(max(end, 1)));
      }
      __syncwarp();
      tensormap_publish(maps.out + x, s_map[wp]);
      __syncwarp();
    }
    return;
  }
  const TileListSpec& l = blockIdx.x == 0 ? l0 : l1;
  const int heads = l.heads, rows_per_block = l.rows_per_block, by_keys = l.by_keys, descending = l.descending,
            max_nblk = l.max_nblk;
  TileEntry* out = l.out;
  const int64_t bound = l.bound;
  __shared__ int64_t shared_start[kSharedSeqs];
  int64_t* seq_start = num_seqs <= kSharedSeqs ? shared_start : scratch;
  if (zero_word != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *zero_word = 0;
  __shared__ int bins[kMaxListBlocks + 1];          // sequences per block count, then cursors
  __shared__ long long bin_start[kMaxListBlocks + 1];  // first entry of each block count
  __shared__ long long warp_sum[kThreads / 32];
  const int tid = static_cast<int>(threadIdx.x);
  const int nb = max_nblk + 1;
  for (int b = tid; b < nb; b += kThreads) bins[b] = 0;
  __syncthreads();
  auto nblk_of = [&](int s) -> int {
    const int* cu = by_keys ? cu_k : cu_q;
    const int len = cu[s + 1] - cu[s];
    const int n = len > 0 ? (len + rows_per_block - 1) / rows_per_block : 0;
    return n < max_nblk ? n : max_nblk;  // max_nblk bounds every sequence (checked on the host)
  };
  for (int s = tid; s < num_seqs; s += kThreads) {
    const int n = nblk_of(s);
    if (n > 0) atomicAdd(&bins[n], 1);
  }
  __syncthreads();
  // bin_start[b] = entries of all block counts above b: a scan from b = nb-1 down.
  // Each thread sums a contiguous chunk of bins; the chunk sums are scanned by warp
  // and over the warps (one thread's scan took most of the kernel: 11 us against 4).
  const int chunk = (nb + kThreads - 1) / kThreads;
  const int b_hi = nb - 1 - tid * chunk;  // this thread's chunk, from the top
  long long acc = 0;
  for (int k = 0; k < chunk; ++k) {
    const int b = b_hi - k;
    if (b < 1) break;
    acc += static_cast<long long>(bins[b]) * b * heads;
  }
  long long inc = acc;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, d);
    if ((tid & 31) >= d) inc += v;
  }
  if ((tid & 31) == 31) warp_sum[tid >> 5] = inc;
  __syncthreads();
  acc = inc - acc;
  for (int w = 0; w < (tid >> 5); ++w) acc += warp_sum[w];
  for (int k = 0; k < chunk; ++k) {
    const int b = b_hi - k;
    if (b < 0) break;
    bin_start[b] = acc;
    if (b >= 1) acc += static_cast<long long>(bins[b]) * b * heads;
  }
  __syncthreads();
  const long long total = bin_start[0];  // all real entries (block count 0 adds none)
  for (int b = tid; b < nb; b += kThreads) bins[b] = 0;  // now cursors
  __syncthreads();
  for (int s = tid; s < num_seqs; s += kThreads) {
    const int n = nblk_of(s);
    seq_start[s] = n > 0 ? bin_start[n] + static_cast<long long>(atomicAdd(&bins[n], 1)) * n * heads : -1;
  }
  __syncthreads();
  // few sequences: several warps each; two lanes per entry, 16 bytes each
  constexpr int kWarps = kThreads / 32;
  const int team = num_seqs < kWarps ? kWarps / max(num_seqs, 1) : 1;
  const int lane = tid & 31, warp = tid >> 5;
  for (int s = warp / team; s < num_seqs; s += kWarps / team) {
    const long long st = seq_start[s];
    if (st < 0) continue;
    const int n = nblk_of(s);
    const int q_start = cu_q[s], k_start = cu_k[s];
    const int4 rows = make_int4(q_start, cu_q[s + 1] - q_start, k_start, cu_k[s + 1] - k_start);
    static_assert(offsetof(TileEntry, head) == 16 && offsetof(TileEntry, seq) == 24, "an entry's two halves");
    for (int u = warp % team * 32 + lane; u < 2 * n * heads; u += team * 32) {
      const int i = u >> 1;
      if (st + i >= bound) break;  // offsets that overrun total rows
      const int h = i / n, k = i % n;
      reinterpret_cast<int4*>(out)[2 * (st + i) + (u & 1)] =
          (u & 1) ? make_int4(h, descending ? n - 1 - k : k, s, 0) : rows;
    }
  }
  for (long long i = total + tid; i < bound; i += kThreads) {
    reinterpret_cast<int4*>(out)[2 * i] = make_int4(0, 0, 0, 0);
    reinterpret_cast<int4*>(out)[2 * i + 1] = make_int4(0, 0, -1, 0);
  }
}

}  // namespace sched

cudaError_t launch_tile_lists(const int* cu_q, const int* cu_k, int num_seqs, const TileListSpec* specs, int n,
                              int64_t* scratch, uint32_t* zero_word, const SeqMaps& maps, cudaStream_t stream) {
  static_assert(sizeof(CUtensorMap) == 128, "a warp copies a map, four bytes a lane");
  if (num_seqs < 0 || n < 0 || n > 2 || maps.n < 0 || maps.n > kMaxSeqMaps || (maps.n > 0 && maps.out == nullptr) ||
      (reinterpret_cast<uintptr_t>(maps.out) & 127u))
    return cudaErrorInvalidValue;
  for (int i = 0; i < n; ++i)
    if (specs[i].max_nblk < 0 || specs[i].max_nblk > kMaxListBlocks || specs[i].rows_per_block <= 0)
      return cudaErrorInvalidValue;
  // more sequences than shared memory holds starts for: one list after another in the scratch
  const int per_launch = num_seqs <= sched::kSharedSeqs ? n : std::min(n, 1);
  const int64_t map_warps = static_cast<int64_t>(num_seqs) * maps.n;
  const int map_blocks = static_cast<int>(std::min<int64_t>((map_warps + sched::kThreads / 32 - 1) / (sched::kThreads / 32), 152));
  int i = 0;
  do {
    const int blocks = per_launch + (i == 0 ? map_blocks : 0);
    if (blocks == 0) break;
    const TileListSpec l0 = n > 0 ? specs[i] : TileListSpec{}, l1 = n > 0 ? specs[i + per_launch - 1] : TileListSpec{};
    sched::tile_list_kernel<<<blocks, sched::kThreads, 0, stream>>>(cu_q, cu_k, num_seqs, l0, l1, per_launch, scratch,
                                                                   zero_word, maps);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    i += per_launch;
  } while (i < n);
  return cudaSuccess;
}

}  // namespace gb300
