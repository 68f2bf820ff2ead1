// attn_prefix.cu -- the tensor cores' kernel (mq_attn_tc.cuh) over shared prefixes
// (attn_shared.cu), and the join of those and what is behind them.
#include "mq_attn_tc.cuh"

namespace mq {

cudaError_t launch_attn_prefix(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    return launch_tc_of<kAttnPrefix>(c, p, grid, status, s);
}

cudaError_t set_attn_prefix_attributes() { return set_tc_attributes<kAttnPrefix>(); }

}  // namespace mq
