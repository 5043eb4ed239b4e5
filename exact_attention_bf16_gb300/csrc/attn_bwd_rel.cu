// Backward variants with a learned relative position bias (rel_bias.cuh).
#include "attn_bwd_rel.cuh"

namespace gb300 {

cudaError_t launch_bwd_dkdv_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  return a.rel.wide ? launch_bwd_dkdv_rel_wide(d_qk, d_v, tq, tk, tv, tdo, a, stream)
                    : bwd::dkdv_rel<kModRelBias>(d_qk, d_v, tq, tk, tv, tdo, a, stream);
}

cudaError_t launch_bwd_dq_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream) {
  return a.rel.wide ? launch_bwd_dq_rel_wide(d_qk, d_v, tq, tk, tv, tdo, a, stream)
                    : bwd::dq_rel<kModRelBias>(d_qk, d_v, tq, tk, tv, tdo, a, stream);
}

}  // namespace gb300
