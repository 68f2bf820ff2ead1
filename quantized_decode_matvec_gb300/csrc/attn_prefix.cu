// attn_prefix.cu -- the tensor cores' kernel (mq_attn_tc.cuh) over shared prefixes
// (attn_shared.cu), and the join of those and what is behind them.
#include "mq_attn_tc.cuh"

namespace mq {

namespace {

// The join takes 32 rows of a row block of a group, and 32 of a head's values, a lane per row: the parts that the
// prefixes' kernel's CTAs left (or, of a block that one CTA finished, its rows), and what the sequences' own keys gave,
// which lies by row too.  With a running maximum, so that a part's values need not wait for the maxima of the others.

// the row block that a CTA of either kernel is for, before anything is read that another kernel writes; false: none.
// Whoever comes after this kernel takes its end for the call's, so every CTA of it waits for the kernels before, those
// without rows too: where no group has any (no pages, no tokens) there are no others.
__device__ __forceinline__ bool join_block(const AttnParams& p, int* grp_s, AttnSegment* g, int* group)
{
    if (threadIdx.x == 0) *grp_s = -1;
    __syncthreads();
    AttnGroup q;
    bool bad;
    for (int k = threadIdx.x; k < p.sh.n_groups; k += blockDim.x)
        if (attn_group(p, k, &q, &bad)) {
            const int64_t at = int64_t(blockIdx.x) - (int64_t(q.t0) * p.group / kPrefixRows + k);
            if (at >= 0 && at * kPrefixRows < int64_t(q.T) * p.group) *grp_s = k;
        }
    __syncthreads();
    const int k = *grp_s;
    if (k < 0) return false;
    (void)attn_group(p, k, &q, &bad);
    g->t0 = q.t0, g->T = q.T, g->head = blockIdx.y;
    g->row0 = int(int64_t(blockIdx.x) - (int64_t(q.t0) * p.group / kPrefixRows + k)) * kPrefixRows;
    *group = k;
    return true;
}

// a row's parts
template <int D>
struct JoinParts {
    const AttnParams& p;
    int4 b;  // the block: first CTA, CTAs, slot of the first
    int64_t place;
    int row, d0;
    __device__ __forceinline__ int count() const { return b.y < 2 ? 2 : b.y + 1; }  // the own keys' first
    // maximum, sum and 32 values of part c
    __device__ __forceinline__ void load(int c, float* m, float* l, float4 (&x)[8]) const
    {
        if (c == 0 || b.y < 2) {
            const AttnRows& from = c == 0 ? p.sh.own : p.sh.prefix;
            const float2 ml = __ldcg(from.ml + place);
            const float4* const src = reinterpret_cast<const float4*>(from.o + place * D + d0);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __ldcg(src + i);
            *m = ml.x, *l = ml.y;
            return;
        }
        const float* const slot = p.parts + (int64_t(b.x + c - 1) * 2 + (c == 1 ? b.z : 0)) * attn_slot_floats(kPrefixRows, D);
        const float4* const src = reinterpret_cast<const float4*>(slot + 2 * kPrefixRows) + d0 / 4 * kPrefixRows + row;
        *m = __ldcg(slot + row) - kTcShift;
        *l = __ldcg(slot + kPrefixRows + row);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __ldcg(src + i * kPrefixRows);
    }
};

struct JoinSum {
    float m = kLowest, l = 0.0f, o[32] = {};
    float gone = 0.0f;  // or what a part says why it has no result
    __device__ __forceinline__ void add(float mc, float lc, const float4 (&x)[8])
    {
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
};

// whether the sequence of a row was not skipped: one that was left the row as it had been
__device__ __noinline__ bool join_row_there(const AttnParams& p, int tok)
{
    for (int s = 0; s < p.c.n_seqs; ++s) {
        AttnSeq e;
        bool wrong;
        if (attn_seq<kAttnOwn>(p, s, &e, &wrong) && e.skip > 0 && tok >= e.t0 && tok - e.t0 < e.T) return true;
    }
    return false;
}

// Few parts: a warp takes them one after the other.
constexpr int kFewWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kFewWarps) attn_shared_join_few_kernel(const AttnParams p, unsigned* status)
{
    __shared__ int grp_s;
    AttnSegment g;
    int k;
    if (!join_block(p, &grp_s, &g, &k)) {
        griddep_wait();
        return;
    }
    const int z = int(blockIdx.z) * kFewWarps + int(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int slab = z / (D / 32) * 32, rows = min(kPrefixRows, g.T * p.group - g.row0);
    const int row = min(slab + lane, rows - 1);
    JoinParts<D> parts = {p, {}, attn_place(p, g, g.row0 + row), row, z % (D / 32) * 32};
    griddep_wait();
    parts.b = __ldcg(p.sh.blocks + attn_block(p, k, g.t0, g.row0, g.head));
    const uint2 flags = __ldcg(reinterpret_cast<const uint2*>(p.sh.abort));
    // a wait ran out: nothing of the call's outputs is known to be whole; or nothing was done
    if (flags.x || (flags.y & kAttnBadOrder) || slab >= rows) return;
    JoinSum sum;
    for (int c = 0; c < parts.count(); ++c) {
        float m, l;
        float4 x[8];
        parts.load(c, &m, &l, x);
        sum.add(m, l, x);
    }
    if (slab + lane >= rows) return;
    if (sum.gone < 0.0f) {
        if (sum.gone == kAttnBadPage) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    if (flags.y && !join_row_there(p, g.t0 + attn_row_token(p, g.row0 + row))) return;
    tc_emit(p, g, g.row0 + row, D, parts.d0, sum.o, sum.l == 0.0f ? 0.0f : 1.0f / sum.l);
}

// Many parts: the warps of a CTA take them in turn, their sums meet in shared memory, where a thread takes four values
// of a row.  Bound by the latency of one or two rounds of loads from L2.
constexpr int kManyWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kManyWarps) attn_shared_join_kernel(const AttnParams p, unsigned* status)
{
    constexpr int W = kManyWarps;
    __shared__ int grp_s;
    __shared__ float m_s[W][32], l_s[W][32];
    __shared__ float o_s[W][32][33];  // [warp][value][row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slab = int(blockIdx.z) / (D / 32) * 32, d0 = int(blockIdx.z) % (D / 32) * 32;
    AttnSegment g;
    int k;
    const bool any = join_block(p, &grp_s, &g, &k);
    const int rows = any ? min(kPrefixRows, g.T * p.group - g.row0) : 0;
    if (slab >= rows) {
        griddep_wait();
        return;
    }
    const int row = min(slab + lane, rows - 1);
    JoinParts<D> parts = {p, {}, attn_place(p, g, g.row0 + row), row, d0};
    griddep_wait();
    parts.b = __ldcg(p.sh.blocks + attn_block(p, k, g.t0, g.row0, g.head));
    const uint2 flags = __ldcg(reinterpret_cast<const uint2*>(p.sh.abort));
    if (flags.x || (flags.y & kAttnBadOrder)) return;
    const int n = parts.count();
    JoinSum own;
    for (int c = warp; c < n; c += W) {
        float m, l;
        float4 x[8];
        parts.load(c, &m, &l, x);
        own.add(m, l, x);
    }
    m_s[warp][lane] = own.m;
    l_s[warp][lane] = own.gone < 0.0f ? own.gone : own.l;
#pragma unroll
    for (int i = 0; i < 32; ++i) o_s[warp][i][lane] = own.o[i];
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
        if (flags.y && there) there = join_row_there(p, g.t0 + attn_row_token(p, g.row0 + slab + r));
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
    const unsigned blocks = unsigned(rows / kPrefixRows + p.sh.n_groups), pieces = slabs * unsigned(c.head_dim / 32);
    // Many parts where there are few blocks for the SMs: 8 blocks of some 10 parts, 19 of a row: 3 and 5 us more for
    // four warps to a CTA than for eight; few where there are many: 95 blocks of 2 or 3 parts.
    if (int64_t(blocks) * c.n_kv_heads * 4 < p.sh.sms) {
        const dim3 grid(blocks, unsigned(c.n_kv_heads), pieces);
        return c.head_dim == 128
                   ? attn_launch_pdl(attn_shared_join_kernel<128>, grid, 32 * kManyWarps, 0, p, status, s)
                   : attn_launch_pdl(attn_shared_join_kernel<64>, grid, 32 * kManyWarps, 0, p, status, s);
    }
    const dim3 grid(blocks, unsigned(c.n_kv_heads), (pieces + kFewWarps - 1) / kFewWarps);
    return c.head_dim == 128 ? attn_launch_pdl(attn_shared_join_few_kernel<128>, grid, 32 * kFewWarps, 0, p, status, s)
                             : attn_launch_pdl(attn_shared_join_few_kernel<64>, grid, 32 * kFewWarps, 0, p, status, s);
}

cudaError_t set_attn_prefix_attributes() { return set_tc_attributes<kAttnPrefix>(); }

}  // namespace mq
