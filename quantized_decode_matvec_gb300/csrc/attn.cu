// attn.cu -- the attention calls: which kernel takes them, their workspace, and
// the kernels for few query rows (mq_attn_rows.cuh) over all of a sequence's keys.
#include "mq_attn_rows.cuh"

namespace mq {

// Workspace: what the join kernels read of the CTAs, the counters, the words of the calls with shared prefixes, parts.
// Where each begins goes by the device alone, so a call finds the counters at zero whatever cache, sequences and rows
// the call before had, and whichever of the two calls it was.
size_t attn_words_offset(int num_sms)
{
    return (size_t(num_sms) * (kAttnSharedBytes + sizeof(unsigned)) + 127) / 128 * 128;
}
size_t attn_parts_offset(int num_sms) { return attn_words_offset(num_sms) + 128; }

// The most query rows of a key/value head that the warp kernels take.  16 rows, 8 key/value heads of 128, here and by
// attn_tc.cu: one sequence of 300 tokens, f16 11.6 and 11.7 us, q8_0 11.9 and 11.9; of 16000 25.3 and 25.8, 23.2 and
// 26.5; 16 of 100 to 3000 29 and 30, 27 and 34; 4 of 30000 84 and 86, 64 and 94.  Seven rows, 4 heads, one sequence of
// 300: 9.3 and 11.5, 9.2 and 11.8; 4 of 30000: 44 and 51, 30 and 55.
constexpr int kWarpRows = 16;

size_t attn_workspace_bytes(const mq_kv_cache& c, int n_heads, int max_tokens, int num_sms)
{
    const int RT = n_heads / c.n_kv_heads * max_tokens > kWarpRows ? attn_tc_rows() : kWarpRows;
    return attn_parts_offset(num_sms) + size_t(num_sms) * 2 * attn_slot_floats(RT, c.head_dim) * sizeof(float);
}

int attn_rows_for(int rows) { return rows <= 8 ? 8 : rows <= kWarpRows ? kWarpRows : attn_tc_rows(); }

AttnParams attn_params(const mq_kv_cache& cache, const mq_attn_args& a, void* ws, int num_sms)
{
    AttnParams p = {};
    p.a = a;
    p.c = kv_view(cache);
    p.group = a.n_heads / cache.n_kv_heads;
    p.group_inv = uint32_t((0x100000000ull + p.group - 1) / p.group);
    p.scale_log2 = float(double(a.scale) * 1.4426950408889634);
    p.shared = static_cast<int4*>(ws);
    p.counters = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + size_t(num_sms) * kAttnSharedBytes);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + attn_parts_offset(num_sms));
    p.limit_ns = uint64_t(fault_policy() == FAULT_NONE ? 2000 : 50) * 1000000ull;
    p.withhold = fault_policy() == FAULT_WITHHOLD_TILE;
    return p;
}

cudaError_t launch_attn(const mq_kv_cache& cache, const mq_attn_args& a, void* ws, int num_sms, unsigned* status,
                        cudaStream_t s)
{
    const AttnParams p = attn_params(cache, a, ws, num_sms);
    const int rows = p.group * a.max_tokens, RT = attn_rows_for(rows);
    // no more CTAs than the bounds allow units
    const int64_t most = int64_t(cache.n_seqs) * ((int64_t(a.max_len) + kKvPage - 1) / kKvPage) * cache.n_kv_heads *
                         ((rows + RT - 1) / RT);
    const int grid = int(most < 1 ? 1 : most < num_sms ? most : num_sms);
    if (RT > kWarpRows) return launch_attn_tc(cache, p, grid, status, s);
    return RT == 8 ? launch_rows_nt<1, kAttnAll>(cache, p, grid, status, s)
                   : launch_rows_nt<2, kAttnAll>(cache, p, grid, status, s);
}

cudaError_t set_attn_attributes(int max_smem)
{
    (void)max_smem;
    cudaError_t e = set_rows_attributes<kAttnAll>();
    if (e == cudaSuccess) e = set_attn_tc_attributes();
    return e;
}

}  // namespace mq
