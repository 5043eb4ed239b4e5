// Backward variants with a learned relative position bias (rel_bias.cuh): the
// dK/dV and dQ kernels of bwd_kernels.cuh, dense or tile-list, also with shared
// K/V heads; the dQ kernel sums the bias's gradient.
#include "bwd_kernels.cuh"

namespace gb300 {

cudaError_t launch_bwd_dkdv_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  using namespace bwd;
  if (a.rel.by_place == nullptr) return cudaErrorInvalidValue;
  if (a.kv_group > 1) {  // shared K/V heads
    if (d_qk == 64 && d_v == 64) return launch_dkdv_t<64, 64, false, kModRelBias, false, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 128 && d_v == 128) return launch_dkdv_wide<false, kModRelBias, true>(tq, tk, tv, tdo, a, stream);
    if (d_qk == 192 && d_v == 128) return launch_dkdv_t<192, 128, false, kModRelBias, false, true>(tq, tk, tv, tdo, a, stream);
  }
  if (d_qk == 64 && d_v == 64) return launch_dkdv_t<64, 64, false, kModRelBias>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 128 && d_v == 128) return launch_dkdv_wide<false, kModRelBias>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 192 && d_v == 128) return launch_dkdv_t<192, 128, false, kModRelBias>(tq, tk, tv, tdo, a, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_bwd_dq_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  using namespace bwd;
  if (a.rel.by_place == nullptr) return cudaErrorInvalidValue;
  if (d_qk == 64 && d_v == 64) return launch_dq_t<64, 64, false, kModRelBias>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 128 && d_v == 128) return launch_dq_t<128, 128, false, kModRelBias>(tq, tk, tv, tdo, a, stream);
  if (d_qk == 192 && d_v == 128) return launch_dq_t<192, 128, false, kModRelBias>(tq, tk, tv, tdo, a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace gb300
