// attn_shared.cu -- attention of a batch whose sequences share the pages of a
// prefix in groups, each prefix attended once for all of its group's tokens.
//
// With the prefix's keys P and a sequence's own keys S of a query row,
//   m = max(m_P, m_S),  l = l_P e^(m_P - m) + l_S e^(m_S - m),  O alike,  out = O / l
// so the two can be attended apart.  Three kernels:
//   own     the keys behind the prefix, sequence by sequence, by the kernels that
//           a call without shared prefixes takes, which leave m, l and O by row;
//   prefix  the tokens of a group as the query rows of one sequence, 256 at a
//           time on the tensor cores: a page is read once per 256 rows of a
//           key/value head where mq_attn_tree reads it once per sequence;
//   join    the prefix's parts and the own result of every row, and its output.
// The prefixes' kernel runs beside the own keys' on the SMs that those leave
// (programmatic dependence; attn_prefix_sms shares them out): neither reads what
// the other writes, and each costs about 10 us of latencies however little it has
// to do.  Where the own keys' parts are joined by a kernel, that comes behind the
// prefixes' kernel: in front of it its waiting CTAs held the SMs' shared memory.
// Measured (28 heads on 4 of 128, q8_0, with a q8_0 output's expansion in torch):
// 64 sequences behind 8192 tokens 44 us (39 alone, where mq_attn_tree takes 98; 66
// one kernel after the other, with a slower join), 4 behind 1000 19 (22.7); f16, 32
// heads on 8: 126 behind three of up to 20011 tokens, trees of up to 7, 238 (252).
#include "mq_attn.cuh"

namespace mq {

namespace {

size_t up(size_t n) { return (n + 127) / 128 * 128; }

struct SharedLayout {
    size_t parts, blocks, own_ml, own_o, pre_ml, pre_o, bytes;
};

// Words that a call finds as the call before left them (the abort word, the counters of the own keys' kernels) lie in
// the part that mq_attn_tree's workspace has too; everything else is written before it is read in every call.
SharedLayout shared_layout(const mq_kv_cache& c, int n_heads, int64_t n_tokens, int max_tokens, int64_t n_groups, int num_sms)
{
    SharedLayout w;
    const int D = c.head_dim, group = n_heads / c.n_kv_heads;
    const size_t rows = size_t(n_tokens) * n_heads;
    w.parts = up(attn_workspace_bytes(c, n_heads, max_tokens, num_sms));  // which the own keys' kernels use
    w.blocks = up(w.parts + size_t(num_sms) * 2 * attn_slot_floats(kPrefixRows, D) * sizeof(float));
    w.own_ml = up(w.blocks + (size_t(n_tokens) * group / kPrefixRows + n_groups + 1) * c.n_kv_heads * sizeof(int4));
    w.own_o = up(w.own_ml + rows * sizeof(float2));
    w.pre_ml = up(w.own_o + rows * D * sizeof(float));
    w.pre_o = up(w.pre_ml + rows * sizeof(float2));
    w.bytes = up(w.pre_o + rows * D * sizeof(float));
    return w;
}

}  // namespace

size_t attn_shared_workspace_bytes(const mq_kv_cache& c, int n_heads, int64_t n_tokens, int max_tokens, int64_t n_groups,
                                   int num_sms)
{
    return shared_layout(c, n_heads, n_tokens, max_tokens, n_groups, num_sms).bytes;
}

cudaError_t launch_attn_shared(const mq_kv_cache& cache, const mq_attn_args& a, const mq_attn_groups& g, void* ws,
                               int num_sms, unsigned* status, cudaStream_t s)
{
    uint8_t* const w = static_cast<uint8_t*>(ws);
    const SharedLayout at = shared_layout(cache, a.n_heads, a.n_tokens, a.max_tokens, g.n_groups, num_sms);
    if (g.n_groups == 0 || g.max_pages == 0) return launch_attn(cache, a, w, num_sms, status, s);
    AttnParams p = attn_params(cache, a, w, num_sms);
    p.sh.grp_start = g.grp_start, p.sh.grp_pages = g.grp_pages;
    p.sh.n_groups = g.n_groups, p.sh.max_pages = g.max_pages;
    p.sh.abort = reinterpret_cast<unsigned*>(w + attn_words_offset(num_sms));
    p.sh.blocks = reinterpret_cast<int4*>(w + at.blocks);
    p.sh.own = AttnRows{reinterpret_cast<float2*>(w + at.own_ml), reinterpret_cast<float*>(w + at.own_o)};
    p.sh.prefix = AttnRows{reinterpret_cast<float2*>(w + at.pre_ml), reinterpret_cast<float*>(w + at.pre_o)};

    const int rows = p.group * a.max_tokens, RT = attn_rows_for(rows);
    const int64_t most = int64_t(cache.n_seqs) * ((int64_t(a.max_len) + kKvPage - 1) / kKvPage) * cache.n_kv_heads *
                         ((rows + RT - 1) / RT);
    const int grid = int(most < 1 ? 1 : most < num_sms ? most : num_sms);
    const int64_t blocks = int64_t(a.n_tokens) * p.group / kPrefixRows + g.n_groups;
    const int64_t units = blocks * cache.n_kv_heads * g.max_pages;
    const int prefix_grid = int(units < num_sms ? units : num_sms);
    // f16: a page of a block of up to 128 rows takes two thirds of the time of one of 256 (one CTA's stretches of equal
    // pages 137 and 201 us); q8_0: the same, since the conversion of its codes is
    p.sh.full = cache.type == MQ_TYPE_F16 ? 3 : 1;
    p.sh.part = cache.type == MQ_TYPE_F16 ? 2 : 1;
    p.sh.sms = num_sms, p.sh.prefix_grid = prefix_grid, p.sh.own_rows = RT;
    cudaError_t e = RT > 16 ? launch_attn_own_tc(cache, p, grid, status, s)
                            : launch_attn_own_rows(cache, p, RT, grid, status, s);
    if (e != cudaSuccess) return e;
    AttnParams pre = p;
    pre.parts = reinterpret_cast<float*>(w + at.parts);
    if ((e = launch_attn_prefix(cache, pre, prefix_grid, status, s)) != cudaSuccess) return e;
    e = RT > 16 ? launch_attn_own_tc_join(cache, p, grid, status, s)
                : launch_attn_own_rows_join(cache, p, RT, grid, status, s);
    return e != cudaSuccess ? e : launch_attn_shared_join(cache, pre, status, s);
}

cudaError_t set_attn_shared_attributes()
{
    cudaError_t e = set_attn_own_rows_attributes();
    if (e == cudaSuccess) e = set_attn_own_tc_attributes();
    if (e == cudaSuccess) e = set_attn_prefix_attributes();
    return e;
}

}  // namespace mq
