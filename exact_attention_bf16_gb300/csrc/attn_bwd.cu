// Backward launchers (the dK/dV and dQ kernels are in bwd_kernels.cuh), the
// D = rowsum(dO * O) pass, the zero fill and the block-list transpose.
#include <cuda_bf16.h>

#include "bwd_kernels.cuh"

namespace gb300 {
namespace bwd {

// D of a row of a sequence (dense: a call) of at most kFewKeys keys, as sum_j P_ij (dO_i . v_j) with P from the LSE, all
// in fp32. The same number as dO_i . O_i in exact arithmetic, but O comes rounded to bf16, and its error d is the same in
// all dS_ij = P_ij (dO_i . v_j - D_i): dQ_i is off by d sum_j P_ij k_j, d up to 2^-8 |dO_i| |O_i|, beside a dQ_i that
// shrinks as the v_j of its keys differ less from their mean O_i. Over sequences of one and two tokens dQ and dK came out
// 5.0e-3 from the exact ones (norms), now below 2.9e-3; from 9 keys on it is at most 3.1e-3 from the rounded O, too. Which
// rows are taken depends on their sequence alone, so that a sequence has the same gradients in every batch.
// Run by the eight lanes l = 0 .. 7 of the row, each with an eighth of the columns (one key each instead left seven lanes
// idle where there is one key, and took 37 us for 29,000 rows); all rows of a warp are of the same unit. Row i (of the
// unit), head h; every lane returns the sum.
__device__ __forceinline__ float few_keys_d(const BwdArgs& a, const FewKeys& t, const Unit& U, int i, int h, int l) {
  auto dot8 = [](const __nv_bfloat16* x, const __nv_bfloat16* y, float sum) {
    const uint4 xv = *reinterpret_cast<const uint4*>(x), yv = *reinterpret_cast<const uint4*>(y);
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, yw[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 xf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&xw[e]));
      const float2 yf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&yw[e]));
      sum = fmaf(xf.x, yf.x, sum);
      sum = fmaf(xf.y, yf.y, sum);
    }
    return sum;
  };
  const int64_t row = U.q_start + i;
  const int pos = i - U.nq + U.nk, hk = h / a.kv_group;  // the row's position among the keys
  const float lse = a.lse[U.b * a.lse_sb + h * a.lse_sh + row];
  const int keys = lse == -INFINITY ? 0 : (a.causal ? min(U.nk, pos + 1) : U.nk);
  const __nv_bfloat16* q = t.q + U.b * t.q_sb + row * t.q_sn + h * t.q_sh;
  const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.dout) + U.b * a.do_sb + row * a.do_sn + h * a.do_sh;
  float acc = 0.f;
  for (int j = 0; j < U.nk; ++j) {
    const __nv_bfloat16* k = t.k + U.b * t.k_sb + static_cast<int64_t>(U.k_start + j) * t.k_sn + hk * t.k_sh;
    const __nv_bfloat16* v = t.v + U.b * t.v_sb + static_cast<int64_t>(U.k_start + j) * t.v_sn + hk * t.v_sh;
    float x = 0.f, y = 0.f;
    for (int c = 8 * l; c < t.d_qk; c += 64) x = dot8(q + c, k + c, x);
    for (int c = 8 * l; c < t.d_v; c += 64) y = dot8(g + c, v + c, y);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if (a.score_mod == kModSoftcap) x = a.mod_b * tanh_scaled(x, a.mod_k2);
    if (a.score_mod == kModAlibi) x -= fabsf(a.alibi_slopes[h] * a.inv_scale * static_cast<float>(j - pos));
    if (j < keys) acc = fmaf(exp2f(fmaf(x, a.scale_log2, -lse * 1.4426950408889634f)), y, acc);
  }
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
  return acc;
}

// Whether few_keys_d is for this unit (offsets past the tensors are not followed). Not with a relative position bias, whose dQ
// kernel takes D from P and dP itself.
__device__ __forceinline__ bool few_keys(const BwdArgs& a, const Unit& U) {
  return a.score_mod != kModRelBias && U.nk >= 1 && U.nk <= kFewKeys && U.q_start >= 0 && U.k_start >= 0 && U.q_start + U.nq <= a.seqlen_q &&
         U.k_start + U.nk <= a.seqlen_k;
}

// D of calls whose rows all see few keys. Latency-bound: four rows a warp. Block x takes units x, x + gridDim.x, ..., its
// rows shared by the blocks along y.
__global__ void __launch_bounds__(256) few_keys_dsum_kernel(const BwdArgs a, const FewKeys t) {
  const int l = static_cast<int>(threadIdx.x & 7u);
  for (int unit = static_cast<int>(blockIdx.x); unit < a.num_units; unit += static_cast<int>(gridDim.x)) {
    const Unit U = unit_bounds(a, unit);
    if (!few_keys(a, U)) continue;
    const int64_t rows = static_cast<int64_t>(U.nq) * a.heads;
    for (int64_t r0 = blockIdx.y * 32 + (threadIdx.x >> 5) * 4; r0 < rows; r0 += gridDim.y * 32) {
      const int64_t r = r0 + ((threadIdx.x >> 3) & 3u), at = min(r, rows - 1);
      const int i = static_cast<int>(at / a.heads), h = static_cast<int>(at % a.heads);
      const float d = few_keys_d(a, t, U, i, h, l);
      if (r < rows && l == 0) a.dsum[U.b * a.lse_sb + h * a.lse_sh + U.q_start + i] = d;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // behind the tile lists' kernel: over before this one is
}

// ===========================================================================
// Preprocess: D = rowsum(dO * O). HBM-bound: DV / 8 lanes share a row, each
// loading 16 bytes of O and of dO per access (rows and head slices start on
// 16-byte boundaries, as the TMA tensor maps already require).
// ===========================================================================
// PACKED: a block takes `chunk` rows side by side and then, where sequences of few keys
// lie in them, replaces those sequences' D by few_keys_d's. (A choice per row in the
// loop cost the rows of longer sequences 40% of its time, a pass of its own behind this
// one 1 us of every call.) A row's token and head are stepped from pass to pass: with
// two divisions a row the pass was bound by its instructions (8 sequences of 2048, 32
// heads, d = 128, the backward: 938 us, 922 so).
constexpr int kPackedBlocks = 6;  // per SM: at 8 few_keys_d spills (3000 sequences of 1 to 30 tokens, the backward: 1550 us, 1621)
template <int DV, bool PACKED>
__global__ void __launch_bounds__(256, PACKED ? kPackedBlocks : 8) preprocess_kernel(const BwdArgs a, const __grid_constant__ FewKeys t, int64_t chunk) {
  constexpr int LPR = DV / 8;    // lanes per row
  constexpr int RPW = 32 / LPR;  // rows per warp
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, l = lane % LPR;
  auto dot8 = [](const uint4& x, const uint4& y) {
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 xf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&xw[e]));
      const float2 yf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&yw[e]));
      acc = fmaf(xf.x, yf.x, acc);
      acc = fmaf(xf.y, yf.y, acc);
    }
#pragma unroll
    for (int s = LPR / 2; s > 0; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    return acc;
  };
  const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(a.o) + 8 * l;
  const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.dout) + 8 * l;
  const int64_t all = static_cast<int64_t>(a.batch) * a.seqlen_q * a.heads;
  const int64_t begin = PACKED ? blockIdx.x * chunk : 0, rows = PACKED ? min(all, begin + chunk) : all;
  if constexpr (PACKED) {
    // two rows in flight
    constexpr int STEP = 8 * RPW;
    const int di = STEP / a.heads, dh = STEP - di * a.heads;
    int64_t r = begin + (threadIdx.x >> 5) * RPW + sub;
    int i = static_cast<int>(r / a.heads), h = static_cast<int>(r - static_cast<int64_t>(i) * a.heads);
    for (int64_t r0 = r - sub; r0 < rows; r0 += 2 * STEP) {
      uint4 ov[2], gv[2];
      int64_t at[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        at[u] = -1;
        ov[u] = gv[u] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          at[u] = h * a.lse_sh + i;
          ov[u] = *reinterpret_cast<const uint4*>(o + i * a.o_sn + h * a.o_sh);
          gv[u] = *reinterpret_cast<const uint4*>(g + i * a.do_sn + h * a.do_sh);
        }
        r += STEP, i += di, h += dh;
        if (h >= a.heads) h -= a.heads, ++i;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float d = dot8(ov[u], gv[u]);
        if (at[u] >= 0 && l == 0) a.dsum[at[u]] = d;
      }
    }
  } else {
    const int64_t warp0 = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    for (int64_t r0 = warp0 * RPW; r0 < rows; r0 += nwarps * RPW) {
      const int64_t r = r0 + sub;
      uint4 ov = make_uint4(0, 0, 0, 0), gv = ov;
      int h = 0, i = 0, b = 0;
      if (r < rows) {
        h = static_cast<int>(r % a.heads);
        const int64_t bi = r / a.heads;
        i = static_cast<int>(bi % a.seqlen_q);
        b = static_cast<int>(bi / a.seqlen_q);
        ov = *reinterpret_cast<const uint4*>(o + b * a.o_sb + i * a.o_sn + h * a.o_sh);
        gv = *reinterpret_cast<const uint4*>(g + b * a.do_sb + i * a.do_sn + h * a.do_sh);
      }
      const float d = dot8(ov, gv);
      if (r < rows && l == 0) a.dsum[b * a.lse_sb + h * a.lse_sh + i] = d;
    }
  }
  if constexpr (PACKED) {
    __syncthreads();  // the D above are written
    const int first = static_cast<int>(begin / a.heads), last = static_cast<int>((rows - 1) / a.heads);  // tokens
    int unit = 0;  // the last sequence that begins at or before `first`
    for (int e = a.num_units; unit + 1 < e;) {
      const int m = (unit + e) / 2;
      if (__ldg(a.cu_q + m) <= first) unit = m;
      else e = m;
    }
    // 32 sequences are looked at together (a step captured for many has a run of empty ones), by every warp alike
    for (bool more = true; more; unit += 32) {
      const int mine = unit + lane;
      const bool in = mine < a.num_units && __ldg(a.cu_q + mine) <= last;
      bool few = false;
      if (in) {
        const Unit U = unit_bounds(a, mine);
        few = U.nq > 0 && few_keys(a, U);
      }
      more = __all_sync(0xffffffffu, in);
      for (uint32_t left = __ballot_sync(0xffffffffu, few); left != 0; left &= left - 1) {
        const Unit U = unit_bounds(a, unit + __ffs(left) - 1);
        const int64_t r_end = min(rows, static_cast<int64_t>(U.q_start + U.nq) * a.heads);
        for (int64_t r0 = max(begin, static_cast<int64_t>(U.q_start) * a.heads) + (threadIdx.x >> 5) * 4; r0 < r_end; r0 += 32) {
          const int64_t r = r0 + (lane >> 3), at = min(r, r_end - 1);
          const int i = static_cast<int>(at / a.heads), h = static_cast<int>(at % a.heads);
          const float d = few_keys_d(a, t, U, i - U.q_start, h, lane & 7);
          if (r < r_end && (lane & 7) == 0) a.dsum[h * a.lse_sh + i] = d;
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // behind the tile lists' kernel: over before this one is
}

// Zero rows: dQ (all queries) and/or dK, dV (all keys).
__global__ void zero_kernel(void* base, int64_t sb, int64_t sn, int64_t sh, int nb, int nrows, int heads, int d) {
  const int64_t total = static_cast<int64_t>(nb) * nrows * heads;
  for (int64_t r = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; r < total;
       r += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int h = static_cast<int>(r % heads);
    const int64_t bi = r / heads;
    const int i = static_cast<int>(bi % nrows);
    const int b = static_cast<int>(bi / nrows);
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + b * sb + i * sn + h * sh;
    for (int c = 0; c < d; ++c) p[c] = __float2bfloat16_rn(0.f);
  }
}

// Transposed block lists: one warp per (list set, key block n) scans the
// query blocks in 32-wide groups, ascending, and appends those whose list
// holds n (a block listed twice counts once). Deterministic: no atomics, fixed
// order. n_sets is 1 (lists shared by every (batch, head)) or batch * heads.
__global__ void transpose_lists_kernel(BwdArgs a, int n_kb, int n_sets) {
  const int64_t w = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) >> 5;
  const int lane = static_cast<int>(threadIdx.x & 31u);
  if (w >= static_cast<int64_t>(n_kb) * n_sets) return;  // whole warps
  const int64_t set = w / n_kb;
  const int n = static_cast<int>(w % n_kb);
  const int* cnt = a.kv_count + set * a.n_qb256;
  const int* idx = a.kv_index + set * a.n_qb256 * a.max_kv;
  int* q_index = const_cast<int*>(a.q_index) + w * a.n_qb256;
  int count = 0;
  for (int b0 = 0; b0 < a.n_qb256; b0 += 32) {
    const int b = b0 + lane;
    bool hit = false;
    if (b < a.n_qb256) {
      int c = cnt[b];
      c = c < 0 ? 0 : (c > a.max_kv ? a.max_kv : c);
      for (int j = 0; j < c && !hit; ++j) hit = idx[static_cast<int64_t>(b) * a.max_kv + j] == n;
    }
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (hit) q_index[count + __popc(m & ((1u << lane) - 1u))] = b;
    count += __popc(m);
  }
  if (lane == 0) const_cast<int*>(a.q_count)[w] = count;
}


}  // namespace bwd

cudaError_t launch_bwd_preprocess(int d_v, const BwdArgs& a, const FewKeys& t, bool early, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.batch) * a.seqlen_q * a.heads;
  if (rows == 0) return cudaSuccess;
  if (d_v != 64 && d_v != 128) return cudaErrorInvalidValue;
  const int64_t per_block = 8 * (d_v == 64 ? 4 : 2);  // 8 warps, each 32 / (d_v / 8) rows per pass
  const int64_t passes = (rows + per_block - 1) / per_block;
  if (a.cu_q != nullptr) {  // one wave of blocks
    const int64_t chunk = (passes + 152 * bwd::kPackedBlocks - 1) / (152 * bwd::kPackedBlocks) * per_block;
    const unsigned blocks = static_cast<unsigned>((rows + chunk - 1) / chunk);
    auto kern = d_v == 64 ? bwd::preprocess_kernel<64, true> : bwd::preprocess_kernel<128, true>;
    if (early) return launch_early(kern, dim3(blocks), 256, 0, stream, a, t, chunk);
    kern<<<blocks, 256, 0, stream>>>(a, t, chunk);
    return cudaGetLastError();
  }
  const unsigned blocks = static_cast<unsigned>(passes < 16384 ? passes : 16384);
  auto kern = d_v == 64 ? bwd::preprocess_kernel<64, false> : bwd::preprocess_kernel<128, false>;
  if (early) return launch_early(kern, dim3(blocks), 256, 0, stream, a, t, int64_t{0});
  kern<<<blocks, 256, 0, stream>>>(a, t, int64_t{0});
  return cudaGetLastError();
}

cudaError_t launch_bwd_few_keys_dsum(const BwdArgs& a, const FewKeys& t, bool early, cudaStream_t stream) {
  if (a.num_units < 1 || a.seqlen_q < 1) return cudaSuccess;
  constexpr int kBlocks = 152 * 4;
  const int gx = a.num_units < kBlocks ? a.num_units : kBlocks;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(kBlocks / gx));
  if (early) return launch_early(bwd::few_keys_dsum_kernel, grid, 256, 0, stream, a, t);
  bwd::few_keys_dsum_kernel<<<grid, 256, 0, stream>>>(a, t);
  return cudaGetLastError();
}

cudaError_t launch_bwd_dkdv(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  if (a.kv_count != nullptr && (a.cu_q != nullptr || a.q_count == nullptr || a.q_index == nullptr))
    return cudaErrorInvalidValue;
  if (a.score_mod != kModNone) return launch_bwd_dkdv_mod(d_qk, d_v, tq, tk, tv, tdo, a, stream);
  if (a.kv_count != nullptr) {
    if (d_qk == 64 && d_v == 64) return bwd::launch_dkdv_t<64, 64, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 128 && d_v == 128) return bwd::launch_dkdv_wide<true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 192 && d_v == 128) return bwd::launch_dkdv_t<192, 128, true>(tq, tk, tv, tdo, a, stream);
    return cudaErrorInvalidValue;
  }
  if (a.kv_group > 1) {  // shared K/V heads
    if (d_qk == 64 && d_v == 64)
      return bwd::launch_dkdv_t<64, 64, false, kModNone, false, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 128 && d_v == 128) return bwd::launch_dkdv_wide<false, kModNone, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 192 && d_v == 128)
      return bwd::launch_dkdv_t<192, 128, false, kModNone, false, true>(tq, tk, tv, tdo, a, stream);
    return cudaErrorInvalidValue;
  }
  if (d_qk == 64 && d_v == 64) return bwd::launch_dkdv_t<64, 64, false>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 128 && d_v == 128) return bwd::launch_dkdv_wide<false>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 192 && d_v == 128) return bwd::launch_dkdv_t<192, 128, false>(tq, tk, tv, tdo, a, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_bwd_transpose_lists(const BwdArgs& a, int n_kb, cudaStream_t stream) {
  if (n_kb <= 0) return cudaSuccess;
  const int n_sets = a.lists_per_head ? a.batch * a.heads : 1;
  const int64_t threads = static_cast<int64_t>(n_kb) * n_sets * 32;
  const int64_t blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  bwd::transpose_lists_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a, n_kb, n_sets);
  return cudaGetLastError();
}

cudaError_t launch_bwd_dq(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  if (a.kv_count != nullptr && a.cu_q != nullptr) return cudaErrorInvalidValue;
  if (a.score_mod != kModNone) return launch_bwd_dq_mod(d_qk, d_v, tq, tk, tv, tdo, a, stream);
  if (a.kv_count != nullptr) {
    if (d_qk == 64 && d_v == 64) return bwd::launch_dq_t<64, 64, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 128 && d_v == 128) return bwd::launch_dq_t<128, 128, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 192 && d_v == 128) return bwd::launch_dq_t<192, 128, true>(tq, tk, tv, tdo, a, stream);
    return cudaErrorInvalidValue;
  }
  if (d_qk == 64 && d_v == 64) return bwd::launch_dq_t<64, 64, false>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 128 && d_v == 128) return bwd::launch_dq_t<128, 128, false>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 192 && d_v == 128) return bwd::launch_dq_t<192, 128, false>(tq, tk, tv, tdo, a, stream);
  return cudaErrorInvalidValue;
}

namespace bwd {

// Split-key dQ: dQ (bf16, strided) = scale * sum_r dq_part[r], the ranges added
// in ascending order (so every call gives the same bits); one thread per 8
// elements of a (batch, head, row).
template <int D>
__global__ void dq_merge_kernel(const BwdArgs a) {
  constexpr int UPR = D / 8;
  const int64_t rows = static_cast<int64_t>(a.batch) * a.heads * a.seqlen_q;  // ((b * heads + h) * seqlen_q + row)
  const int64_t units = rows * UPR;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < units;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int c = static_cast<int>(i % UPR);
    const int64_t rh = i / UPR;
    const int row = static_cast<int>(rh % a.seqlen_q);
    const int64_t bh = rh / a.seqlen_q;
    const int h = static_cast<int>(bh % a.heads), b = static_cast<int>(bh / a.heads);
    const float* src = a.dq_part + rh * D + 8 * c;
    float4 x = __ldg(reinterpret_cast<const float4*>(src)), y = __ldg(reinterpret_cast<const float4*>(src) + 1);
    for (int r = 1; r < a.dq_split; ++r) {
      const float4* pr = reinterpret_cast<const float4*>(src + r * rows * D);
      const float4 u = __ldg(pr), w = __ldg(pr + 1);
      x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
      y = make_float4(y.x + w.x, y.y + w.y, y.z + w.z, y.w + w.w);
    }
    const float sc = a.scale;
    const uint4 o = make_uint4(pack_bf16x2(x.x * sc, x.y * sc), pack_bf16x2(x.z * sc, x.w * sc),
                               pack_bf16x2(y.x * sc, y.y * sc), pack_bf16x2(y.z * sc, y.w * sc));
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dq) + b * a.dq_sb + static_cast<int64_t>(row) * a.dq_sn +
                         h * a.dq_sh + 8 * c;
    *reinterpret_cast<uint4*>(dst) = o;
  }
}

}  // namespace bwd

cudaError_t launch_bwd_dq_merge(const BwdArgs& a, int d_qk, cudaStream_t stream) {
  if (a.dq_split < 2 || a.dq_part == nullptr || a.cu_q != nullptr) return cudaErrorInvalidValue;
  const int64_t units = static_cast<int64_t>(a.batch) * a.heads * a.seqlen_q * (d_qk / 8);
  if (units == 0) return cudaSuccess;
  const int64_t want = (units + 255) / 256;
  const unsigned blocks = static_cast<unsigned>(want < 152 * 16 ? want : 152 * 16);
  if (d_qk == 64) bwd::dq_merge_kernel<64><<<blocks, 256, 0, stream>>>(a);
  else if (d_qk == 128) bwd::dq_merge_kernel<128><<<blocks, 256, 0, stream>>>(a);
  else if (d_qk == 192) bwd::dq_merge_kernel<192><<<blocks, 256, 0, stream>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

namespace bwd {

// One thread per 8 elements of a (key row, K/V head): the parts added in ascending
// order, so that every call gives the same bits. Rows behind the last sequence of a
// packed batch are left alone, as the kernels leave them.
__global__ void dkv_merge_kernel(const BwdArgs a, int d_qk, int d_v) {
  const int width = d_qk + d_v, upr = width / 8;
  const int64_t rows = static_cast<int64_t>(a.batch) * a.seqlen_k, units = rows * a.heads_kv * upr;
  const int64_t last = a.cu_k != nullptr ? a.cu_k[a.num_units] : rows;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < units;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int c = 8 * static_cast<int>(i % upr);
    const int64_t rh = i / upr, row = rh / a.heads_kv;
    const int h = static_cast<int>(rh % a.heads_kv);
    if (row >= last) continue;
    const float* src = a.dkv_part + rh * width + c;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int r = 0; r < a.dkv_split; ++r) {
      const float4* pr = reinterpret_cast<const float4*>(src + r * rows * a.heads_kv * width);
      const float4 u = __ldg(pr), w = __ldg(pr + 1);
      x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
      y = make_float4(y.x + w.x, y.y + w.y, y.z + w.z, y.w + w.w);
    }
    const float sc = c < d_qk ? a.scale : 1.f;
    const int64_t b = row / a.seqlen_k, n = row % a.seqlen_k;
    __nv_bfloat16* dst = c < d_qk ? static_cast<__nv_bfloat16*>(a.dk) + b * a.dk_sb + n * a.dk_sn + h * a.dk_sh + c
                                  : static_cast<__nv_bfloat16*>(a.dv) + b * a.dv_sb + n * a.dv_sn + h * a.dv_sh + c - d_qk;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x.x * sc, x.y * sc), pack_bf16x2(x.z * sc, x.w * sc),
                                                pack_bf16x2(y.x * sc, y.y * sc), pack_bf16x2(y.z * sc, y.w * sc));
  }
}

}  // namespace bwd

cudaError_t launch_bwd_dkv_merge(const BwdArgs& a, int d_qk, int d_v, cudaStream_t stream) {
  if (a.dkv_split < 2 || a.dkv_part == nullptr) return cudaErrorInvalidValue;
  const int64_t units = static_cast<int64_t>(a.batch) * a.seqlen_k * a.heads_kv * ((d_qk + d_v) / 8);
  const int64_t want = (units + 255) / 256;
  bwd::dkv_merge_kernel<<<static_cast<unsigned>(want < 152 * 16 ? want : 152 * 16), 256, 0, stream>>>(a, d_qk, d_v);
  return cudaGetLastError();
}

cudaError_t launch_bwd_zero(const BwdArgs& a, int d_qk, int d_v, bool zero_dq, bool zero_dkdv, cudaStream_t stream) {
  auto go = [&](void* p, int64_t sb, int64_t sn, int64_t sh, int nrows, int heads, int d) -> cudaError_t {
    const int64_t total = static_cast<int64_t>(a.batch) * nrows * heads;
    if (total == 0) return cudaSuccess;
    const int blocks = static_cast<int>(total / 256 + 1 < 4096 ? total / 256 + 1 : 4096);
    bwd::zero_kernel<<<blocks, 256, 0, stream>>>(p, sb, sn, sh, a.batch, nrows, heads, d);
    return cudaGetLastError();
  };
  cudaError_t e = cudaSuccess;
  if (zero_dq) e = go(a.dq, a.dq_sb, a.dq_sn, a.dq_sh, a.seqlen_q, a.heads, d_qk);
  if (e == cudaSuccess && zero_dkdv) e = go(a.dk, a.dk_sb, a.dk_sn, a.dk_sh, a.seqlen_k, a.heads_kv, d_qk);
  if (e == cudaSuccess && zero_dkdv) e = go(a.dv, a.dv_sb, a.dv_sn, a.dv_sh, a.seqlen_k, a.heads_kv, d_v);
  return e;
}

}  // namespace gb300
