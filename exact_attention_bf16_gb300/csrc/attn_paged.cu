// Attention of packed new tokens over a paged KV cache (attn_fwd_paged).
//
// O_i = sum_j softmax_j(a_ij) v_j over the visible keys of query i, a_ij =
// scale q_i . k_j, in one pass over the keys with a running maximum m, sum l
// and accumulator (log2 units): for a new block of keys with maximum m',
//   alpha = 2^(m - max(m, m')), l = l alpha + sum 2^(a - m), acc = acc alpha + 2^(a - m) v.
#include "kernels.h"
#include "ptx_sm100.cuh"
#include "score_mod.cuh"

namespace gb300 {
namespace paged {

// One warp per (query row, head): 32 keys at a time, one per lane for the
// logits, then one after another for the PV sums (lane l holds columns l, l +
// 32, ...). Every sum is fp32. Correct for every case; each warp reads its keys
// alone, so it is bound by L2 and issue, not by HBM or the tensor cores.
template <int DQK, int DV>
__global__ void __launch_bounds__(128) paged_row_kernel(const PagedArgs a) {
  __shared__ float sq[4][DQK];
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int64_t r = blockIdx.x * 4ll + warp;
  if (r >= static_cast<int64_t>(a.total_q) * a.heads) return;
  const int t = static_cast<int>(r / a.heads), h = static_cast<int>(r % a.heads), hk = h / a.kv_group;
  int lo = 0, hi = a.num_seqs;  // the request whose rows hold t
  if (t < a.cu_q[0] || t >= a.cu_q[a.num_seqs]) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int i = t - a.cu_q[lo], nq = min(a.cu_q[lo + 1] - a.cu_q[lo], a.max_q);
  if (i >= nq) return;
  const int nk = max(0, min(a.seqlens_k[lo], a.max_keys));
  const int lim = a.causal ? min(nk, i + (nk - nq) + 1) : nk;
  const int qpos = i + (nk - nq);
  const int* table = a.block_table + lo * a.block_table_stride;
  for (int c = lane; c < DQK; c += 32) sq[warp][c] = __bfloat162float(a.q[t * a.q_row + h * a.q_head + c]);
  __syncwarp();
  const float slope = a.score_mod == kModAlibi ? a.alibi_slopes[h] * a.inv_scale : 0.f;
  float m = -INFINITY, l = 0.f, acc[DV / 32];
#pragma unroll
  for (int c = 0; c < DV / 32; ++c) acc[c] = 0.f;
  for (int j0 = 0; j0 < lim; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    const __nv_bfloat16* vrow = nullptr;
    if (j < lim) {
      const int page = table[j >> a.page_shift];
      if (page >= 0 && page < a.num_pages) {
        const int64_t row = j & (a.page_size - 1);
        const __nv_bfloat16* krow = a.k + page * a.k_page + row * a.k_row + hk * a.k_head;
        vrow = a.v + page * a.v_page + row * a.v_row + hk * a.v_head;
        float dot = 0.f;
        for (int c = 0; c < DQK; c += 2) {
          const float2 kf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(krow + c));
          dot = fmaf(kf.x, sq[warp][c], dot);
          dot = fmaf(kf.y, sq[warp][c + 1], dot);
        }
        if (a.score_mod == kModSoftcap) dot = a.mod_b * tanh_scaled(dot, a.mod_k2);
        if (a.score_mod == kModAlibi) dot -= fabsf(slope) * fabsf(static_cast<float>(j - qpos));
        s = dot * a.scale_log2;
      }
    }
    float mx = s;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if (mx == -INFINITY) continue;
    const float mn = fmaxf(m, mx), alpha = exp2f(m - mn);
    m = mn;
    const float p = exp2f(s - mn);
    l = l * alpha + p;
#pragma unroll
    for (int c = 0; c < DV / 32; ++c) acc[c] *= alpha;
    for (int u = 0; u < 32; ++u) {
      const float pu = __shfl_sync(0xffffffffu, p, u);
      const __nv_bfloat16* vu = reinterpret_cast<const __nv_bfloat16*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vrow), u));
      if (vu == nullptr) continue;
#pragma unroll
      for (int c = 0; c < DV / 32; ++c) acc[c] = fmaf(pu, __bfloat162float(vu[lane + 32 * c]), acc[c]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < DV / 32; ++c) a.o[t * a.o_row + h * a.o_head + lane + 32 * c] = __float2bfloat16_rn(acc[c] * inv);
  if (lane == 0)
    a.lse[static_cast<int64_t>(h) * a.total_q + t] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace paged

cudaError_t launch_fwd_paged(int d_qk, int d_v, const PagedArgs& a, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(a.total_q) * a.heads + 3) / 4;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(blocks);
  if (d_qk == 64 && d_v == 64) paged::paged_row_kernel<64, 64><<<g, 128, 0, stream>>>(a);
  else if (d_qk == 128 && d_v == 128) paged::paged_row_kernel<128, 128><<<g, 128, 0, stream>>>(a);
  else if (d_qk == 192 && d_v == 128) paged::paged_row_kernel<192, 128><<<g, 128, 0, stream>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace gb300
