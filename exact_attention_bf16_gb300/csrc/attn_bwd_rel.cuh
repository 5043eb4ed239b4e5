// The backward with a relative position bias, by head size (attn_bwd_rel.cu, attn_bwd_rel_wide.cu): the
// dK/dV and dQ kernels of bwd_kernels.cuh, dense or tile-list, also with shared
// K/V heads; the dQ kernel sums the bias's gradient.
#pragma once
#include "bwd_kernels.cuh"

namespace gb300 {
namespace bwd {

template <int MOD>
cudaError_t dkdv_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  if (a.rel.by_place == nullptr) return cudaErrorInvalidValue;
  if (a.kv_group > 1) {  // shared K/V heads
    if (d_qk == 64 && d_v == 64) return launch_dkdv_t<64, 64, false, MOD, false, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 128 && d_v == 128) return launch_dkdv_wide<false, MOD, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 192 && d_v == 128) return launch_dkdv_t<192, 128, false, MOD, false, true>(tq, tk, tv, tdo, a, stream);
  }
  if (d_qk == 64 && d_v == 64) return launch_dkdv_t<64, 64, false, MOD>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 128 && d_v == 128) return launch_dkdv_wide<false, MOD>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 192 && d_v == 128) return launch_dkdv_t<192, 128, false, MOD>(tq, tk, tv, tdo, a, stream);
  return cudaErrorInvalidValue;
}

template <int MOD>
cudaError_t dq_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  if (a.rel.by_place == nullptr) return cudaErrorInvalidValue;
  if (d_qk == 64 && d_v == 64) return launch_dq_t<64, 64, false, MOD>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 128 && d_v == 128) return launch_dq_t<128, 128, false, MOD>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 192 && d_v == 128) return launch_dq_t<192, 128, false, MOD>(tq, tk, tv, tdo, a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace bwd
}  // namespace gb300
