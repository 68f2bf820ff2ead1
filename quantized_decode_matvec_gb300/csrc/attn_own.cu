// attn_own.cu -- the kernels for few query rows over the keys behind a shared
// prefix (attn_shared.cu).
#include "mq_attn_rows.cuh"

namespace mq {

cudaError_t launch_attn_own_rows(const mq_kv_cache& c, const AttnParams& p, int RT, int grid, unsigned* status,
                                 cudaStream_t s)
{
    return RT == 8 ? launch_rows_nt<1, kAttnOwn>(c, p, grid, status, s) : launch_rows_nt<2, kAttnOwn>(c, p, grid, status, s);
}

cudaError_t launch_attn_own_rows_join(const mq_kv_cache& c, const AttnParams& p, int RT, int grid, unsigned* status,
                                      cudaStream_t s)
{
    if (RT == 8) return cudaSuccess;  // the CTA that comes last has joined
    return c.head_dim == 128 ? launch_rows_join<128, 2, kAttnOwn>(p, grid, status, s)
                             : launch_rows_join<64, 2, kAttnOwn>(p, grid, status, s);
}

cudaError_t set_attn_own_rows_attributes() { return set_rows_attributes<kAttnOwn>(); }

}  // namespace mq
