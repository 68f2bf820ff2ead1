// mq_attn.cuh -- what the attention kernels share: the split of a call's work
// over the CTAs, its partial results in the workspace, and the output rows.
//
// The work of a call is a line of units.  Sequence s, key/value head h and
// block b of its query rows (token * group + head of the group) form a group;
// a group's units are its pages of kKvPage keys, and the groups follow one another in the order (s, h, b).  CTA c of N takes the units
// [c*W/N, (c+1)*W/N) of all W, so every CTA has the same number of pages
// whatever the lengths are, and lengths are read on the device only.  A CTA's
// stretch of a group is a segment.  A group that lies in one CTA is finished
// there; otherwise each of its CTAs leaves its segment's maxima, sums and
// unnormalised outputs in the workspace, and the one that arrives last at the
// group's counter joins them in CTA order (so the result does not depend on
// who was last) and returns the counter to zero.
#pragma once

#include <cuda_fp16.h>

#include "mq_internal.h"
#include "mq_kv.cuh"
#include "mq_stream.cuh"
#include "mq_tma.cuh"

namespace mq {

constexpr int kAttnGroupCost = 3;

struct AttnParams {
    mq_attn_args a;
    KvView c;
    int group;           // query heads per key/value head
    float scale_log2;    // scale * log2(e): exp(x) = 2^(x log2 e)
    unsigned* counters;  // one per group
    float* parts;        // two slots of a segment's results per CTA
    uint64_t limit_ns;
};

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

// Called by all threads of the CTA; scratch: an int2 per warp.
__device__ __forceinline__ AttnRange attn_range(const AttnParams& p, int RT, unsigned* status, int2* scratch, int2* at_s)
{
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.c.n_seqs + nthr - 1) / nthr, s0 = min(tid * per, p.c.n_seqs), s1 = min(s0 + per, p.c.n_seqs);
    int2 mine = make_int2(0, 0);  // pages of all groups, groups
    bool any_bad = false;
    for (int s = s0; s < s1; ++s) {
        AttnSeq q;
        bool bad;
        if (attn_seq(p, s, &q, &bad)) {
            const int n = attn_groups(p, q, RT);
            mine.x += n * q.pages;
            mine.y += n;
        }
        any_bad |= bad;
    }
    if (any_bad && blockIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
    int2 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
        if (lane >= o) incl.x += x, incl.y += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    AttnRange r;
    int2 before = make_int2(0, 0), total = before;
    for (int w = 0; w < nthr / 32; ++w) {
        if (w == warp) before = total;
        total.x += scratch[w].x, total.y += scratch[w].y;
    }
    r.cost = total.x > int(gridDim.x) ? kAttnGroupCost : 0;
    r.total = total.x + total.y * r.cost;
    r.ctas = min(r.total, int(gridDim.x));
    const int c = blockIdx.x;
    r.quot = r.ctas ? r.total / r.ctas : 0;
    r.rem = r.total - r.quot * r.ctas;
    r.first = c < r.ctas ? r.begin(c) : r.total;
    r.last = c < r.ctas ? r.begin(c + 1) : r.total;
    int at = before.x + incl.x - mine.x + (before.y + incl.y - mine.y) * r.cost;
    if (r.first >= at && r.first < at + mine.x + mine.y * r.cost) {
        for (int s = s0; s < s1; ++s) {
            AttnSeq q;
            bool bad;
            if (!attn_seq(p, s, &q, &bad)) continue;
            const int u = attn_groups(p, q, RT) * (q.pages + r.cost);
            if (r.first < at + u) {
                *at_s = make_int2(s, at);
                break;
            }
            at += u;
        }
    }
    __syncthreads();
    r.seq = at_s->x;
    r.seq_first = at_s->y;
    return r;
}

// one segment, as the producer describes it to the other roles
struct AttnSegment {
    int seq, t0, T, ctx;
    int head, row0;   // key/value head; first query row of the block
    int page0, n;     // its pages page0 .. page0 + n - 1; n = 0: the stretch is done
    int group_index;  // of the counters
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
        const int k = (u - w->seq_first) / span;  // group within the sequence
        const int g0 = w->seq_first + k * span, g1 = g0 + q.pages;
        if (u >= g1) {
            u = g0 + span;
            continue;
        }
        g->seq = w->seq;
        g->t0 = q.t0, g->T = q.T, g->ctx = q.ctx;
        g->head = k / blocks;
        g->row0 = (k - g->head * blocks) * RT;
        g->page0 = u - g0;
        g->n = min(g1, w->last) - u;
        const int most = (p.a.max_tokens * p.group + RT - 1) / RT;
        g->group_index = (w->seq * p.c.n_kv_heads + g->head) * most + k - g->head * blocks;
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

// A segment's results in the workspace: m[RT], l[RT] (l < 0 in row 0: the
// segment met a page outside the cache), then RT rows of D outputs.
__host__ __device__ constexpr int64_t attn_slot_floats(int RT, int D) { return int64_t(RT) * (D + 2); }

// one warp writes 32 consecutive outputs (lane l: value d0 + l) of a query row
__device__ __forceinline__ void attn_emit(const AttnParams& p, const AttnSegment& g, int row, int D, int d0, float v)
{
    const int lane = threadIdx.x & 31;
    const int tok = g.t0 + row / p.group, h = g.head * p.group + row % p.group;
    if (p.a.out_type == MQ_TYPE_F16) {
        static_cast<__half*>(p.a.out)[int64_t(tok) * p.a.out_ld + h * D + d0 + lane] = __float2half_rn(v);
    } else {
        float sc;
        const int code = q8_quantize_lane(v, &sc);
        uint8_t* const ob =
            static_cast<uint8_t*>(p.a.out) + (int64_t(tok) * (p.a.n_heads * D / 32) + (h * D + d0) / 32) * kQ8Bytes;
        if (lane == 0) *reinterpret_cast<__half*>(ob) = __float2half_rn(sc);
        ob[2 + lane] = uint8_t(int8_t(code));
    }
}

// a segment's arrival at its group's counter; true in the CTA that came last
// (one thread calls it, after the CTA's results are written and synchronised)
__device__ __forceinline__ bool attn_arrive(const AttnParams& p, const AttnSegment& g)
{
    __threadfence();
    unsigned* const c = p.counters + g.group_index;
    const bool is_last = atomicAdd(c, 1u) == unsigned(g.n_ctas - 1);
    if (is_last) {
        *c = 0;  // nobody else of this call comes back to it
        __threadfence();
    }
    return is_last;
}

}  // namespace mq
