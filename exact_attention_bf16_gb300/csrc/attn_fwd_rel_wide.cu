// The forward with a relative position bias whose table has a wide bucket (RelBias::wide).
#include "attn_fwd_rel.cuh"

namespace gb300 {

cudaError_t launch_fwd_rel_wide(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tv16, const FwdArgs& a, cudaStream_t stream) {
  return fwd::launch_rel<kModRelWide>(d_qk, d_v, tq, tk, tv, tv16, a, stream);
}

}  // namespace gb300
