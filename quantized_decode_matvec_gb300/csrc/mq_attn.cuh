// mq_attn.cuh -- what the attention kernels share: the split of a call's work
// over the CTAs, its partial results in the workspace, and the output rows.
//
// The work of a call is a line of units.  Sequence s, key/value head h and
// block b of its query rows (token * group + head of the group) form a group;
// a group's units are its pages of kKvPage keys and, where the CTAs have more
// than a page each, kAttnGroupCost units for its start and end.  The groups
// follow one another in the order (s, h, b).  CTA c of N takes the units
// [c*W/N, (c+1)*W/N) of all W, so every CTA has the same work whatever the
// lengths are, and lengths are read on the device only.  A CTA's stretch of a
// group is a segment.  A group that lies in one CTA is finished there;
// otherwise each of its CTAs leaves its segment's maxima, sums and
// unnormalised outputs in the workspace, and they are joined in CTA order (so
// the result does not depend on who was last): of up to eight query rows by
// the CTA that comes last to the group's counter, which returns it to zero; of
// more by a kernel behind that all SMs take part in, launched with programmatic
// dependence, to which a group's first CTA describes it.  One sequence of 16000
// tokens, four key/value heads of 128, q8_0, seven rows: 14.7 us joined by the
// last CTA, 16.0 by the kernel; 4000 tokens, eight heads, 16 rows: 20.0 and 17.0.
#pragma once

#include <cuda_fp16.h>

#include "mq_internal.h"
#include "mq_kv.cuh"
#include "mq_stream.cuh"
#include "mq_tma.cuh"

namespace mq {

// In pages.  One query token per sequence, q8_0, D 128, at a cost of 2, 4, 6, 8, 10 and 14: 64 sequences of 128 to 8191
// tokens, 4 key/value heads: 67, 66, 61, 60, 59 and 59 us; 256 of 100 to 1000, 8 heads: 83, 81, 82, 84, 84 and 87; 16
// trees of 16 nodes over 128 to 8000 tokens, 8 heads: 90, 76, 61, 60, 62 and 65.  The entry check's bound on the units
// counts on at most 11.
constexpr int kAttnGroupCost = 8;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^x (x <= 0) as the factor of sums and outputs that a larger maximum scales down.  It does not go to zero: an
// infinite value in a sum stays infinite, where 0 * inf is NaN, and 2^-126 of a finite one is nothing beside the key
// with the maximum.
__device__ __forceinline__ float attn_factor(float x)
{
    return fmaxf(ex2(x), 0x1p-126f);
}

struct AttnParams {
    mq_attn_args a;
    KvView c;
    int group;           // query heads per key/value head
    uint32_t group_inv;  // 2^32 / group rounded up: x / group = umulhi(x, group_inv) for x < 2^16
    float scale_log2;    // scale * log2(e): exp(x) = 2^(x log2 e)
    int4* shared;        // per CTA: the group that it starts and the next one goes on with (attn_shared)
    unsigned* counters;  // one per CTA: arrivals at the group that it starts and the next one goes on with
    float* parts;        // two slots of a segment's results per CTA
    uint64_t limit_ns;
    int withhold;  // test-only: the last page of a CTA's first segment is never delivered
};

// query row r of a sequence is head r % group of the group, of token r / group
__device__ __forceinline__ int attn_row_token(const AttnParams& p, int r)
{
    return p.group == 1 ? r : int(__umulhi(uint32_t(r), p.group_inv));
}

// sequence s as the device data has it; false (and nothing to do) where it is
// empty, *bad where it contradicts the call's bounds or the cache
struct AttnSeq {
    int t0, T, ctx, pages;
};
__device__ __forceinline__ bool attn_seq(const AttnParams& p, int s, AttnSeq* q, bool* bad)
{
    q->t0 = __ldg(p.a.tok_start + s);
    const int64_t T = int64_t(__ldg(p.a.tok_start + s + 1)) - q->t0;
    q->ctx = __ldg(p.a.ctx_len + s);
    const int64_t len = q->ctx + T;
    *bad = q->t0 < 0 || T < 0 || T > p.a.max_tokens || q->t0 + T > p.a.n_tokens ||
           (T > 0 && (q->ctx < 0 || len > p.a.max_len || len > int64_t(p.c.table_ld) * kKvPage));
    q->T = int(T);
    q->pages = int((len + kKvPage - 1) / kKvPage);
    return T > 0 && !*bad;
}

// groups of sequence s with row blocks of RT rows; each has q.pages + (the group cost) units
__device__ __forceinline__ int attn_groups(const AttnParams& p, const AttnSeq& q, int RT)
{
    return p.c.n_kv_heads * ((q.T * p.group + RT - 1) / RT);
}

// The cut of the line, and where this CTA's stretch starts.
struct AttnRange {
    int total, ctas;  // all units; the CTAs that take part (each has a unit at least)
    int quot, rem;    // total / ctas, total % ctas
    int cost;         // units of a group beyond its pages
    int first, last;  // this CTA's units
    int seq;          // sequence that the walk is at, and its first unit
    int seq_first;
    __device__ __forceinline__ int begin(int c) const { return c * quot + min(c, rem); }
    __device__ __forceinline__ int owner(int u) const
    {
        const int longer = rem * (quot + 1);
        return u < longer ? u / (quot + 1) : rem + (u - longer) / quot;
    }
};

// The cut, and where this CTA's stretch starts; called by one whole warp.
__device__ __forceinline__ AttnRange attn_range(const AttnParams& p, int RT, unsigned* status)
{
    const int lane = threadIdx.x & 31, n = gridDim.x, c = blockIdx.x;
    int pages = 0, groups = 0;
    bool any_bad = false;
    for (int s = lane; s < p.c.n_seqs; s += 32) {
        AttnSeq q;
        bool bad;
        if (attn_seq(p, s, &q, &bad)) {
            const int k = attn_groups(p, q, RT);
            pages += k * q.pages;
            groups += k;
        }
        any_bad |= bad;
    }
    if (any_bad && c == 0) atomicOr(status, MQ_DEV_KV_RANGE);
    pages = __reduce_add_sync(0xffffffffu, pages);
    groups = __reduce_add_sync(0xffffffffu, groups);
    AttnRange r;
    r.cost = pages > n ? kAttnGroupCost : 0;
    r.total = pages + groups * r.cost;
    r.ctas = min(r.total, n);
    r.quot = r.ctas ? r.total / r.ctas : 0;
    r.rem = r.total - r.quot * r.ctas;
    r.first = c < r.ctas ? r.begin(c) : r.total;
    r.last = c < r.ctas ? r.begin(c + 1) : r.total;
    r.seq = 0, r.seq_first = 0;
    // the sequence that holds unit r.first, 32 at a time
    for (int s0 = 0; s0 < p.c.n_seqs && r.first < r.last; s0 += 32) {
        AttnSeq q;
        bool bad;
        const int mine = s0 + lane < p.c.n_seqs && attn_seq(p, s0 + lane, &q, &bad)
                             ? attn_groups(p, q, RT) * (q.pages + r.cost) : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, r.first < r.seq_first + incl);
        const int l = past ? __ffs(past) - 1 : 31;
        const int upto = __shfl_sync(0xffffffffu, past ? incl - mine : incl, l);
        r.seq_first += upto;
        r.seq = s0 + l;
        if (past) break;
    }
    return r;
}

// one segment, as the producer describes it to the other roles
struct AttnSegment {
    int seq, t0, T, ctx;
    int head, row0;   // key/value head; first query row of the block
    int page0, n;     // its pages page0 .. page0 + n - 1; n = 0: the stretch is done
    int cta0, n_ctas; // the CTAs that share the group
    int slot0;        // workspace slot of the first of them (the others use 0)
    int slot;         // this CTA's slot
};

// The next segment of a CTA's stretch, which starts at unit *at of sequence
// w->seq or a later one; *at moves past it.  False: there is none.
__device__ __forceinline__ bool attn_next(const AttnParams& p, int RT, AttnRange* w, int* at, AttnSegment* g)
{
    for (int u = *at; u < w->last;) {
        AttnSeq q;
        bool bad;
        const int units = attn_seq(p, w->seq, &q, &bad) ? attn_groups(p, q, RT) * (q.pages + w->cost) : 0;
        if (u >= w->seq_first + units) {
            w->seq_first += units;
            if (++w->seq >= p.c.n_seqs) return false;  // not reached unless the lengths change under the call
            continue;
        }
        const int blocks = (q.T * p.group + RT - 1) / RT, span = q.pages + w->cost;
        const int k = u - w->seq_first < span ? 0 : (u - w->seq_first) / span;  // group within the sequence
        const int g0 = w->seq_first + k * span, g1 = g0 + q.pages;
        if (u >= g1) {
            u = g0 + span;
            continue;
        }
        g->seq = w->seq;
        g->t0 = q.t0, g->T = q.T, g->ctx = q.ctx;
        g->head = blocks == 1 ? k : k / blocks;
        g->row0 = (k - g->head * blocks) * RT;
        g->page0 = u - g0;
        g->n = min(g1, w->last) - u;
        const bool whole = g0 >= w->first && g1 <= w->last;
        g->cta0 = whole ? int(blockIdx.x) : w->owner(g0);
        g->n_ctas = whole ? 1 : w->owner(g1 - 1) - g->cta0 + 1;
        g->slot0 = g0 > w->begin(g->cta0) ? 1 : 0;
        g->slot = u > w->first ? 1 : 0;
        *at = u + g->n;
        return true;
    }
    return false;
}

// A segment's results in the workspace: m[RT], l[RT], then RT rows of D
// outputs.  A negative l says that there are none, and the group stays
// unwritten: the segment met a page outside the cache, or its CTA gave up
// (the slot may hold another call's results then).
__host__ __device__ constexpr int64_t attn_slot_floats(int RT, int D) { return int64_t(RT) * (D + 2); }
constexpr float kAttnBadPage = -1.0f, kAttnGaveUp = -2.0f;

// what the join has to know of a group (n_ctas = 0: nothing to join)
constexpr int kAttnSharedBytes = 32;
__device__ __forceinline__ void attn_shared(const AttnSegment& g, int4 (&s)[2])
{
    s[0] = make_int4(g.t0, g.T, g.head, g.row0);
    s[1] = make_int4(g.n_ctas, g.slot0, 0, 0);
}

// a warp writes rows, four values d .. d + 3 per lane (the eight lanes of a block of 32 lie together)
__device__ __forceinline__ void attn_emit4(const AttnParams& p, const AttnSegment& g, int row, bool there, int D, int d,
                                           float4 v)
{
    const int lane = threadIdx.x & 31;
    const int node = attn_row_token(p, row), h = (g.head - node) * p.group + row;
    const int64_t tok = g.t0 + node;
    if (p.a.out_type == MQ_TYPE_F16) {
        const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
        if (there)
            *reinterpret_cast<uint2*>(static_cast<__half*>(p.a.out) + tok * p.a.out_ld + h * D + d) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        return;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(fabsf(x[i])));
#pragma unroll
    for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Q8Scale s = q8_scale_of(__uint_as_float(top));
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int c;
        if (!q8_code_fast(x[i], s, &c)) c = q8_code_exact(x[i], s.d);
        code |= uint32_t(c & 255) << (8 * i);
    }
    if (!there) return;
    uint16_t* const ob = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.a.out) +
                                                     (tok * (p.a.n_heads * D / 32) + (h * D + d) / 32) * kQ8Bytes);
    if (lane % 8 == 0) ob[0] = __half_as_ushort(__float2half_rn(s.d));
    ob[1 + d % 32 / 2] = uint16_t(code);
    ob[2 + d % 32 / 2] = uint16_t(code >> 16);
}

// a segment's arrival at its group's counter, which is that of the group's first CTA (a CTA is the first of one
// shared group at most: the one that reaches past its stretch); true in the CTA that came last
// (one thread calls it, after the CTA's results are written and synchronised)
__device__ __forceinline__ bool attn_arrive(const AttnParams& p, const AttnSegment& g)
{
    unsigned* const c = p.counters + g.cta0;
    unsigned before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(c) : "memory");
    const bool is_last = before == unsigned(g.n_ctas - 1);
    if (is_last) *c = 0;  // nobody else of this call comes back to it
    return is_last;
}

// barrier over n threads; true for all of them where it was for one
__device__ __forceinline__ bool barrier_any(int id, int n, bool v)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(v)), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

// the join behind the kernel that has just been launched
template <class K>
cudaError_t attn_launch_join(K kernel, dim3 grid, int threads, size_t smem, const AttnParams& p, unsigned* status,
                             cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, status);
}

// many query rows per key/value head (attn_tc.cu): rows of a block there, its launch and set-up
int attn_tc_rows();
cudaError_t launch_attn_tc(const mq_kv_cache& cache, const AttnParams& p, int grid, unsigned* status, cudaStream_t s);
cudaError_t set_attn_tc_attributes();

}  // namespace mq
