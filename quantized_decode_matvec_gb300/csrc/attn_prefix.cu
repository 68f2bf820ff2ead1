// attn_prefix.cu -- the tensor cores' kernel (mq_attn_tc.cuh) over shared prefixes
// (attn_shared.cu), and the join of those and what is behind them.
#include "mq_attn_tc.cuh"

namespace mq {

namespace {

// A CTA per (row block of the groups, key/value head, 32 of its rows and 32 of a head's values).  Its warps take the
// parts of the block in turn, a lane per row: those that the prefixes' kernel's CTAs left (or, of a block that one CTA
// finished, its rows), and what the sequences' own keys gave, which lies by row too.  Each warp keeps a running
// maximum, so that a part's values need not wait for the maxima of the others; then the warps' sums meet in shared
// memory, where a thread takes four values of a row.  Bound by the latency of one round of loads from L2, and behind
// long prefixes of many rows by the parts' bytes.
template <int D, int W>
__global__ void __launch_bounds__(32 * W) attn_shared_join_kernel(const AttnParams p, unsigned* status)
{
    __shared__ int grp_s;
    __shared__ float m_s[W][32], l_s[W][32];
    __shared__ float o_s[W][32][33];  // [warp][value][row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slab = int(blockIdx.z) / (D / 32) * 32, d0 = int(blockIdx.z) % (D / 32) * 32;
    if (threadIdx.x == 0) grp_s = -1;
    __syncthreads();
    AttnGroup q;
    bool bad;
    for (int k = threadIdx.x; k < p.sh.n_groups; k += (32 * W))
        if (attn_group(p, k, &q, &bad)) {
            const int64_t at = int64_t(blockIdx.x) - (int64_t(q.t0) * p.group / kPrefixRows + k);
            if (at >= 0 && at * kPrefixRows < int64_t(q.T) * p.group) grp_s = k;
        }
    __syncthreads();
    const int k = grp_s;
    if (k < 0) return;
    (void)attn_group(p, k, &q, &bad);
    AttnSegment g;
    g.t0 = q.t0, g.T = q.T, g.head = blockIdx.y;
    g.row0 = int(int64_t(blockIdx.x) - (int64_t(q.t0) * p.group / kPrefixRows + k)) * kPrefixRows;
    const int rows = min(kPrefixRows, g.T * p.group - g.row0);
    if (slab >= rows) return;
    const int row = min(slab + lane, rows - 1);
    const int64_t place = attn_place(p, g, g.row0 + row);
    griddep_wait();
    const int4 b = __ldcg(p.sh.blocks + attn_block(p, k, g.t0, g.row0, g.head));
    const uint2 flags = __ldcg(reinterpret_cast<const uint2*>(p.sh.abort));
    if (flags.x) return;  // a wait ran out: nothing of the call's outputs is known to be whole
    const int n = b.y < 2 ? 2 : b.y + 1;  // parts, the own keys' first
    const float* const first = p.parts + (int64_t(b.x) * 2 + b.z) * attn_slot_floats(kPrefixRows, D);
    const float* const others = p.parts + int64_t(b.x) * 2 * attn_slot_floats(kPrefixRows, D);
    float m = kLowest, l = 0.0f, o[32];
    float gone = 0.0f;  // or what a part says why it has no result
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
    for (int c = warp; c < n; c += W) {
        float mc, lc;
        float4 x[8];
        if (c == 0 || b.y < 2) {
            const AttnRows& from = c == 0 ? p.sh.own : p.sh.prefix;
            const float2 ml = __ldcg(from.ml + place);
            const float4* const src = reinterpret_cast<const float4*>(from.o + place * D + d0);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __ldcg(src + i);
            mc = ml.x, lc = ml.y;
        } else {
            const float* const slot = c == 1 ? first : others + int64_t(c - 1) * 2 * attn_slot_floats(kPrefixRows, D);
            const float4* const src = reinterpret_cast<const float4*>(slot + 2 * kPrefixRows) + d0 / 4 * kPrefixRows + row;
            mc = __ldcg(slot + row) - kTcShift;
            lc = __ldcg(slot + kPrefixRows + row);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __ldcg(src + i * kPrefixRows);
        }
        if (lc < 0.0f) gone = gone == kAttnBadPage ? gone : lc;
        const float top = fmaxf(m, mc), f = attn_factor(m - top), fc = attn_factor(mc - top);
        m = top;
        l = fmaf(l, f, lc * fc);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[4 * i] = fmaf(o[4 * i], f, x[i].x * fc);
            o[4 * i + 1] = fmaf(o[4 * i + 1], f, x[i].y * fc);
            o[4 * i + 2] = fmaf(o[4 * i + 2], f, x[i].z * fc);
            o[4 * i + 3] = fmaf(o[4 * i + 3], f, x[i].w * fc);
        }
    }
    m_s[warp][lane] = m;
    l_s[warp][lane] = gone < 0.0f ? gone : l;
#pragma unroll
    for (int i = 0; i < 32; ++i) o_s[warp][i][lane] = o[i];
    __syncthreads();
    const int v4 = threadIdx.x % 8 * 4, nw = min(n, W);
#pragma unroll
    for (int r = threadIdx.x / 8; r < 32; r += (32 * W) / 8) {
        float top = kLowest, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        bool there = slab + r < rows, bad_page = false;
        for (int w = 0; w < nw; ++w) top = fmaxf(top, m_s[w][r]);
        for (int w = 0; w < nw; ++w) {
            const float f = attn_factor(m_s[w][r] - top), lw = l_s[w][r];
            if (lw < 0.0f && there) {
                bad_page |= lw == kAttnBadPage;
                there = false;
            }
            sum = fmaf(lw, f, sum);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(o_s[w][v4 + i][r], f, v[i]);
        }
        if (flags.y && there) {  // rows of a sequence that was skipped hold what was there
            const int tok = g.t0 + attn_row_token(p, g.row0 + slab + r);
            bool found = false;
            for (int s = 0; s < p.c.n_seqs && !found; ++s) {
                AttnSeq e;
                bool wrong;
                found = attn_seq<kAttnOwn>(p, s, &e, &wrong) && e.skip > 0 && tok >= e.t0 && tok - e.t0 < e.T;
            }
            there = found;
        }
        if (bad_page) atomicOr(status, MQ_DEV_KV_RANGE);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        __syncwarp();
        attn_emit4(p, g, g.row0 + min(slab + r, rows - 1), there, D, d0 + v4,
                   make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
    }
}

}  // namespace

cudaError_t launch_attn_prefix(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    return launch_tc_of<kAttnPrefix>(c, p, grid, status, s);
}

cudaError_t launch_attn_shared_join(const mq_kv_cache& c, const AttnParams& p, unsigned* status, cudaStream_t s)
{
    const int64_t rows = int64_t(p.a.n_tokens) * p.group;
    const unsigned slabs = unsigned(((rows < kPrefixRows ? rows : kPrefixRows) + 31) / 32);
    const dim3 grid(unsigned(rows / kPrefixRows + p.sh.n_groups), unsigned(c.n_kv_heads), slabs * unsigned(c.head_dim / 32));
    // Eight warps where a block has many parts, four where it has a few and there are many blocks: 8 blocks of some 10
    // parts and 19 of a row, 3 and 5 us; 95 blocks of 2 or 3 parts 33 and 19 us.
    const bool many = int64_t(grid.x) * grid.y * 4 < p.sh.sms;
#define MQ_JOIN(D, W) attn_launch_pdl(attn_shared_join_kernel<D, W>, grid, 32 * W, 0, p, status, s)
    return c.head_dim == 128 ? (many ? MQ_JOIN(128, 8) : MQ_JOIN(128, 4)) : (many ? MQ_JOIN(64, 8) : MQ_JOIN(64, 4));
#undef MQ_JOIN
}

cudaError_t set_attn_prefix_attributes()
{
    cudaError_t e = set_tc_attributes<kAttnPrefix>();
    // shared memory for as many CTAs as the threads allow
#define MQ_SET(D, W)     \
    if (e == cudaSuccess) \
        e = cudaFuncSetAttribute(attn_shared_join_kernel<D, W>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    MQ_SET(128, 8) MQ_SET(64, 8) MQ_SET(128, 4) MQ_SET(64, 4)
#undef MQ_SET
    return e;
}

}  // namespace mq
