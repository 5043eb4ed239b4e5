// Forward variants with a learned relative position bias (rel_bias.cuh): the
// kernel of fwd_kernel.cuh, dense and tile-list (packed variable length).
#include "attn_fwd_rel.cuh"

namespace gb300 {

cudaError_t launch_fwd_rel(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const CUtensorMap& tv16, const FwdArgs& a, cudaStream_t stream) {
  return a.rel.wide ? launch_fwd_rel_wide(d_qk, d_v, tq, tk, tv, tv16, a, stream)
                    : fwd::launch_rel<kModRelBias>(d_qk, d_v, tq, tk, tv, tv16, a, stream);
}

}  // namespace gb300
