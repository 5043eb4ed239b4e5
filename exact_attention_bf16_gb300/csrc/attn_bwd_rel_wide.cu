// The backward with a relative position bias whose table has a wide bucket (RelBias::wide).
#include "attn_bwd_rel.cuh"

namespace gb300 {

cudaError_t launch_bwd_dkdv_rel_wide(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                     const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  return bwd::dkdv_rel<kModRelWide>(d_qk, d_v, tq, tk, tv, tdo, a, stream);
}

cudaError_t launch_bwd_dq_rel_wide(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  return bwd::dq_rel<kModRelWide>(d_qk, d_v, tq, tk, tv, tdo, a, stream);
}

}  // namespace gb300
