// attn_tc.cu -- the tensor cores' kernel (mq_attn_tc.cuh) over all of a sequence's keys.
#include "mq_attn_tc.cuh"

namespace mq {

int attn_tc_rows() { return kTcRows; }

cudaError_t launch_attn_tc(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    return launch_tc_of<kAttnAll>(c, p, grid, status, s);
}

cudaError_t set_attn_tc_attributes() { return set_tc_attributes<kAttnAll>(); }

}  // namespace mq
