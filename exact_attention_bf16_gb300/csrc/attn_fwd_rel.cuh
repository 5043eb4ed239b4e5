// The forward with a relative position bias, by head size (attn_fwd_rel.cu, attn_fwd_rel_wide.cu).
#pragma once
#include "fwd_kernel.cuh"

namespace gb300 {
namespace fwd {

template <int DQK, int DV, int MOD>
cudaError_t launch_r(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tv16,
                     const FwdArgs& a, cudaStream_t stream) {
  if (a.tiles != nullptr) return launch_e<DQK, DV, 0, false, false, true, MOD>(tq, tk, tv, tv16, a, stream);
  return launch_e<DQK, DV, 0, false, false, false, MOD>(tq, tk, tv, tv16, a, stream);
}

template <int MOD>
cudaError_t launch_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tv16, const FwdArgs& a, cudaStream_t stream) {
  if (a.emu_period != 0 || a.kv_count != nullptr || a.rel.by_place == nullptr) return cudaErrorInvalidValue;
  if (d_qk == 64 && d_v == 64) return launch_r<64, 64, MOD>(tq, tk, tv, tv16, a, stream);
  if (d_qk == 128 && d_v == 128) return launch_r<128, 128, MOD>(tq, tk, tv, tv16, a, stream);
  if (d_qk == 192 && d_v == 128) return launch_r<192, 128, MOD>(tq, tk, tv, tv16, a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fwd
}  // namespace gb300
