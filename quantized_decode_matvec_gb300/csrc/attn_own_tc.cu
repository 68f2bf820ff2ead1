// attn_own_tc.cu -- the tensor cores' kernel (mq_attn_tc.cuh) over the keys behind a shared
// prefix (attn_shared.cu).
#include "mq_attn_tc.cuh"

namespace mq {

cudaError_t launch_attn_own_tc(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    return launch_tc_of<kAttnOwn>(c, p, grid, status, s);
}

cudaError_t launch_attn_own_tc_join(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    return c.head_dim == 128 ? launch_tc_join<128, kAttnOwn>(p, grid, status, s)
                             : launch_tc_join<64, kAttnOwn>(p, grid, status, s);
}

cudaError_t set_attn_own_tc_attributes() { return set_tc_attributes<kAttnOwn>(); }

}  // namespace mq
