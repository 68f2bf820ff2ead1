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

// Which keys a kernel attends over: all of a sequence's; in a call with shared prefixes (attn_shared.cu) a sequence's
// own ones, those behind the pages that its group shares; or those pages, for all tokens of a group's sequences, which
// the kernel takes for one long sequence without a tree.  The last two leave their rows' maxima, sums and unnormalised
// outputs for the join, but for a sequence without shared pages, which the second finishes.
enum { kAttnAll = 0, kAttnOwn = 1, kAttnPrefix = 2 };
constexpr int kPrefixRows = 256;  // query rows of a block (mq_attn_tc.cuh)

// Rows (token * heads + head) in the workspace.  ml: the maximum less the kernel's shift, so that ml.y 2^ml.x is the
// sum whichever kernel it is from; a negative ml.y: there is no result (a page outside the cache).
struct AttnRows {
    float2* ml;
    float* o;  // [rows][D]
};

// what the device's data contradicts: a sequence the call's bounds or its group (it is skipped), or the groups the order
// of grp_start, so that a sequence might lie in two of them (the whole call is skipped)
constexpr int kAttnBadSeq = 1, kAttnBadOrder = 2;

struct AttnShared {
    const int32_t* grp_start;
    const int32_t* grp_pages;
    int n_groups, max_pages;
    int sms, prefix_grid, own_rows;  // SMs that the two kernels share out; the second's CTAs; the first's rows of a block
    int full, part;  // units of a prefix's page in a block of 256 rows, and of up to 128
    unsigned* abort;  // [0]: a wait ran out; [1]: kAttnBadSeq, kAttnBadOrder
    AttnRows own, prefix;
    int4* blocks;   // per row block and key/value head of the groups: first CTA, CTAs, slot of the first
};

struct AttnParams {
    mq_attn_args a;
    KvView c;
    int group;           // query heads per key/value head
    uint32_t group_inv;  // 2^32 / group rounded up: x / group = umulhi(x, group_inv) for x < 2^32 / group
    float scale_log2;    // scale * log2(e): exp(x) = 2^(x log2 e)
    int4* shared;        // per CTA: the group that it starts and the next one goes on with (attn_shared)
    unsigned* counters;  // one per CTA: arrivals at the group that it starts and the next one goes on with
    float* parts;        // two slots of a segment's results per CTA
    uint64_t limit_ns;
    int withhold;  // test-only: the last page of a CTA's first segment is never delivered
    AttnShared sh;  // not kAttnAll
};

// query row r of a sequence is head r % group of the group, of token r / group
__device__ __forceinline__ int attn_row_token(const AttnParams& p, int r)
{
    return p.group == 1 ? r : int(__umulhi(uint32_t(r), p.group_inv));
}

// Group g of the sequences with a shared prefix; false where there is nothing to do for it, *bad where it contradicts
// the call's bounds.
struct AttnGroup {
    int seq0, t0, T, pages;
    int row;  // of the table: that of the first sequence with tokens
};
__device__ __forceinline__ bool attn_group(const AttnParams& p, int g, AttnGroup* q, bool* bad)
{
    q->seq0 = __ldg(p.sh.grp_start + g);
    const int end = __ldg(p.sh.grp_start + g + 1);
    q->pages = __ldg(p.sh.grp_pages + g);
    *bad = q->seq0 < 0 || end < q->seq0 || end > p.c.n_seqs || q->pages < 0 || q->pages > p.sh.max_pages ||
           q->pages > p.c.table_ld;
    q->t0 = q->T = 0, q->row = q->seq0;
    if (*bad) return false;
    q->t0 = __ldg(p.a.tok_start + q->seq0);
    const int64_t T = int64_t(__ldg(p.a.tok_start + end)) - q->t0;
    *bad = q->t0 < 0 || T < 0 || q->t0 + T > p.a.n_tokens;
    q->T = int(T);
    if (!(T > 0 && q->pages > 0 && !*bad)) return false;
    while (q->row + 1 < end && __ldg(p.a.tok_start + q->row + 1) == q->t0) ++q->row;
    return true;
}

// The group of sequence s, or -1: the last that has it.
constexpr int kLaneGroups = 32;  // up to here a warp keeps a group per lane (attn_range)
__device__ __forceinline__ int attn_group_of(const AttnParams& p, int s)
{
    if (p.sh.n_groups <= kLaneGroups) {
        int g = -1;
        for (int k = 0; k < p.sh.n_groups; ++k)
            if (s >= __ldg(p.sh.grp_start + k) && s < __ldg(p.sh.grp_start + k + 1)) g = k;
        return g;
    }
    int lo = 0, hi = p.sh.n_groups;  // the last group that starts at s or before it
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.sh.grp_start + mid) <= s)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo > 0 && s < __ldg(p.sh.grp_start + lo) ? lo - 1 : -1;
}

// Groups in a warp's registers, one per lane: looked up without loads that wait for one another.
struct AttnLaneGroup {
    int seq0, end, t0, T, pages;
    int state;  // 0: nothing to do, 1: there, 2: contradicts the bounds
};
__device__ __forceinline__ AttnLaneGroup attn_lane_group(const AttnParams& p)
{
    AttnLaneGroup l = {};
    const int k = threadIdx.x & 31;
    if (p.sh.n_groups <= kLaneGroups && k < p.sh.n_groups) {
        AttnGroup q;
        bool bad;
        const bool there = attn_group(p, k, &q, &bad);
        l.seq0 = q.seq0, l.end = __ldg(p.sh.grp_start + k + 1);
        l.t0 = q.t0, l.T = q.T, l.pages = q.pages;
        l.state = bad ? 2 : there ? 1 : 0;
    }
    return l;
}

// sequence s as the device data has it (kAttnPrefix: group s as one); false
// (and nothing to do) where it is empty, *bad where it contradicts the call's
// bounds or the cache
struct AttnSeq {
    int t0, T, ctx, pages;
    int row, skip;  // its row of the table; kAttnOwn: pages of the table before its own
};
// its tokens lie in the group's, which the join goes by, and its context reaches past the prefix
__device__ __forceinline__ void attn_own(AttnSeq* q, bool* bad, int state, int t0, int T, int pages)
{
    *bad = state == 2 || (state == 1 && (q->t0 < t0 || q->t0 + int64_t(q->T) > int64_t(t0) + T || q->ctx < pages * kKvPage));
    if (state == 1 && !*bad) {
        q->skip = pages;
        q->ctx -= pages * kKvPage;
    }
}
// by a thread
template <int M>
__device__ __forceinline__ bool attn_seq(const AttnParams& p, int s, AttnSeq* q, bool* bad)
{
    if constexpr (M == kAttnPrefix) {
        AttnGroup g;
        const bool there = attn_group(p, s, &g, bad);
        q->t0 = g.t0, q->T = g.T, q->pages = g.pages, q->ctx = g.pages * kKvPage, q->row = g.row, q->skip = 0;
        return there;
    }
    q->t0 = __ldg(p.a.tok_start + s);
    const int64_t T = int64_t(__ldg(p.a.tok_start + s + 1)) - q->t0;
    q->ctx = __ldg(p.a.ctx_len + s);
    const int64_t len = q->ctx + T;
    *bad = q->t0 < 0 || T < 0 || T > p.a.max_tokens || q->t0 + T > p.a.n_tokens ||
           (T > 0 && (q->ctx < 0 || len > p.a.max_len || len > int64_t(p.c.table_ld) * kKvPage));
    q->T = int(T), q->row = s, q->skip = 0;
    if constexpr (M == kAttnOwn) {
        const int k = T > 0 && !*bad ? attn_group_of(p, s) : -1;
        if (k >= 0) {
            AttnGroup g;
            bool bad_group;
            const bool there = attn_group(p, k, &g, &bad_group);
            attn_own(q, bad, bad_group ? 2 : there, g.t0, g.T, g.pages);
        }
    }
    q->pages = int((q->ctx + T + kKvPage - 1) / kKvPage);
    return T > 0 && !*bad;
}
// by a whole warp, which comes together: every lane its sequence (there: it has one)
template <int M>
__device__ __forceinline__ bool attn_seq(const AttnParams& p, const AttnLaneGroup& lg, int s, bool there, AttnSeq* q,
                                         bool* bad)
{
    *bad = false;
    if (M != kAttnOwn || p.sh.n_groups > kLaneGroups) return there && attn_seq<M>(p, s, q, bad);
    if (there) there = attn_seq<kAttnAll>(p, s, q, bad);
    int k = 0;
    bool in = false;
    for (int i = 0; i < p.sh.n_groups; ++i) {
        const int from = __shfl_sync(0xffffffffu, lg.seq0, i), to = __shfl_sync(0xffffffffu, lg.end, i);
        if (s >= from && s < to) k = i, in = true;
    }
    const int state = __shfl_sync(0xffffffffu, lg.state, k), t0 = __shfl_sync(0xffffffffu, lg.t0, k);
    const int T = __shfl_sync(0xffffffffu, lg.T, k), pages = __shfl_sync(0xffffffffu, lg.pages, k);
    if (there && in) {
        attn_own(q, bad, state, t0, T, pages);
        q->pages = (q->ctx + q->T + kKvPage - 1) / kKvPage;
    }
    return there && !*bad;
}
template <int M>
__device__ __forceinline__ int attn_seqs(const AttnParams& p)
{
    return M == kAttnPrefix ? p.sh.n_groups : p.c.n_seqs;
}

// groups of sequence s with row blocks of RT rows; each has q.pages + (the group cost) units
__device__ __forceinline__ int attn_groups(const AttnParams& p, const AttnSeq& q, int RT)
{
    return p.c.n_kv_heads * ((q.T * p.group + RT - 1) / RT);
}

// kAttnPrefix: a block of up to 128 rows is one tile of the tensor cores, of more two, so a page of a sequence's last
// block may count for less
__device__ __forceinline__ int attn_unit(const AttnParams& p, const AttnSeq& q, int block)
{
    return q.T * p.group - block * kPrefixRows > kPrefixRows / 2 ? p.sh.full : p.sh.part;
}
// units of a key/value head's blocks of sequence s, and of all heads'
template <int M>
__device__ __forceinline__ int attn_head_units(const AttnParams& p, const AttnSeq& q, int RT, int cost)
{
    const int blocks = (q.T * p.group + RT - 1) / RT;
    if (M != kAttnPrefix) return blocks * (q.pages + cost);
    return ((blocks - 1) * p.sh.full + attn_unit(p, q, blocks - 1)) * q.pages + blocks * cost;
}
template <int M>
__device__ __forceinline__ int attn_units(const AttnParams& p, const AttnSeq& q, int RT, int cost)
{
    return p.c.n_kv_heads * attn_head_units<M>(p, q, RT, cost);
}

// The cut of the line, and where this CTA's stretch starts.
struct AttnRange {
    int total, ctas;  // all units; the CTAs that take part (each has a unit at least)
    int quot, rem;    // total / ctas, total % ctas
    int cost;         // units of a group beyond its pages
    int first, last;  // this CTA's units
    int seq;          // sequence that the walk is at, and its first unit
    int seq_first;
    AttnLaneGroup lg; // kAttnOwn
    __device__ __forceinline__ int begin(int c) const { return c * quot + min(c, rem); }
    __device__ __forceinline__ int owner(int u) const
    {
        const int longer = rem * (quot + 1);
        return u < longer ? u / (quot + 1) : rem + (u - longer) / quot;
    }
};

// The SMs of a call with shared prefixes go to both kernels, x of N to the prefixes', such that they end together:
//   d + A / x = B / (N - x)
// in units of a page of the kernel for few rows, 0.45 us; a group is kAttnGroupCost more.  A page of 256 rows on the
// tensor cores takes two units; of the sequences' own keys there, of few rows mostly, about half a one, and a group
// twice as much (1024 groups of 28 rows and 6 pages, f16: 67 us on 152 SMs).  d: what the prefixes' kernel starts later, and takes
// longer to start and to leave its parts.
__device__ __forceinline__ float attn_prefix_sms(const AttnParams& p, int pages, int groups, int pre_pages, int pre_groups)
{
    const bool tc = p.sh.own_rows > 16;
    const float d = 16.0f, N = float(p.sh.sms);
    const float A = 2.0f * (pre_pages / float(p.sh.full) + float(kAttnGroupCost) * pre_groups);
    const float B = (tc ? 0.55f : 1.0f) * pages + (tc ? 2.2f : 1.0f) * kAttnGroupCost * groups;
    const float b = d * N - A - B;
    return (b + sqrtf(b * b + 4.0f * d * A * N)) / (2.0f * d);
}

// What the sequences and the groups come to, formed by all warps of a CTA, 32 sequences each at a time, before
// attn_range (kAttnAll: by the one warp that calls it).
struct AttnTotals {
    int own[(MQ_MAX_SEQS + 31) / 32][2];  // pages and groups of 32 sequences
    int pages, groups, pre_pages, pre_groups, bad;  // (pre_pages: their units; bad: kAttnBadSeq, kAttnBadOrder)
};
template <int M>
__device__ __forceinline__ void attn_totals(const AttnParams& p, AttnTotals* t)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (threadIdx.x == 0) t->pages = t->groups = t->pre_pages = t->pre_groups = t->bad = 0;
    __syncthreads();
    const AttnLaneGroup lg = attn_lane_group(p);
    AttnSeq q;
    bool bad, any_bad = false, order = false;
    for (int k = threadIdx.x; k < p.sh.n_groups; k += blockDim.x)
        order |= __ldg(p.sh.grp_start + k + 1) < __ldg(p.sh.grp_start + k);
    for (int i = warp; 32 * i < p.c.n_seqs; i += warps) {
        int pages = 0, groups = 0;
        if (attn_seq<kAttnOwn>(p, lg, 32 * i + lane, 32 * i + lane < p.c.n_seqs, &q, &bad)) {
            groups = attn_groups(p, q, p.sh.own_rows);
            pages = groups * q.pages;
        }
        any_bad |= bad;
        pages = __reduce_add_sync(0xffffffffu, pages);
        groups = __reduce_add_sync(0xffffffffu, groups);
        if (lane == 0) {
            t->own[i][0] = pages, t->own[i][1] = groups;
            atomicAdd(&t->pages, pages);
            atomicAdd(&t->groups, groups);
        }
    }
    for (int i = warps - 1 - warp; 32 * i < p.sh.n_groups; i += warps) {  // from the last warp on
        int pages = 0, groups = 0;
        if (32 * i + lane < p.sh.n_groups) {
            if (attn_seq<kAttnPrefix>(p, 32 * i + lane, &q, &bad)) {
                groups = attn_groups(p, q, kPrefixRows);
                pages = attn_units<kAttnPrefix>(p, q, kPrefixRows, 0);
            }
            any_bad |= bad;
        }
        pages = __reduce_add_sync(0xffffffffu, pages);
        groups = __reduce_add_sync(0xffffffffu, groups);
        if (lane == 0) {
            atomicAdd(&t->pre_pages, pages);
            atomicAdd(&t->pre_groups, groups);
        }
    }
    if (any_bad || order) atomicOr(&t->bad, (any_bad ? kAttnBadSeq : 0) | (order ? kAttnBadOrder : 0));
    __syncthreads();
}

// The cut, and where this CTA's stretch starts; called by one whole warp.
template <int M>
__device__ __forceinline__ AttnRange attn_range(const AttnParams& p, int RT, const AttnTotals* t, unsigned* status)
{
    const int lane = threadIdx.x & 31, c = blockIdx.x;
    int n = gridDim.x, pages = 0, groups = 0;
    AttnRange r;
    r.lg = AttnLaneGroup{};
    if constexpr (M == kAttnAll) {
        bool any_bad = false;
        for (int s = lane; s < p.c.n_seqs; s += 32) {
            AttnSeq q;
            bool bad;
            if (attn_seq<M>(p, s, &q, &bad)) {
                const int k = attn_groups(p, q, RT);
                pages += k * q.pages;
                groups += k;
            }
            any_bad |= bad;
        }
        if (any_bad && c == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        pages = __reduce_add_sync(0xffffffffu, pages);
        groups = __reduce_add_sync(0xffffffffu, groups);
    } else {
        r.lg = attn_lane_group(p);
        int take = p.sh.sms - int(attn_prefix_sms(p, t->pages, t->groups, t->pre_pages, t->pre_groups) + 0.5f);
        take = t->pre_pages > 0 ? min(max(take, p.sh.sms - p.sh.prefix_grid), p.sh.sms - 1) : p.sh.sms;
        n = min(n, max(M == kAttnOwn ? take : p.sh.sms - take, 1));
        pages = M == kAttnPrefix ? t->pre_pages : t->pages;
        groups = M == kAttnPrefix ? t->pre_groups : t->groups;
        if (t->bad & kAttnBadOrder) pages = groups = 0;
        if (M == kAttnOwn && c == 0 && lane == 0) {
            p.sh.abort[1] = t->bad;  // the join looks closer then
            if (t->bad) atomicOr(status, MQ_DEV_KV_RANGE);
        }
    }
    const int unit = M == kAttnPrefix ? p.sh.full : 1;
    r.cost = pages > n * unit ? kAttnGroupCost * unit : 0;
    r.total = pages + groups * r.cost;
    // a CTA between others that share a group has a page at least
    r.ctas = M == kAttnPrefix ? min(max(r.total / unit, min(r.total, 1)), n) : min(r.total, n);
    r.quot = r.ctas ? r.total / r.ctas : 0;
    r.rem = r.total - r.quot * r.ctas;
    r.first = c < r.ctas ? r.begin(c) : r.total;
    r.last = c < r.ctas ? r.begin(c + 1) : r.total;
    r.seq = 0, r.seq_first = 0;
    // the sequence that holds unit r.first, 32 at a time
    for (int s0 = 0; s0 < attn_seqs<M>(p) && r.first < r.last; s0 += 32) {
        if (M == kAttnOwn) {  // not among these
            const int units = t->own[s0 / 32][0] + t->own[s0 / 32][1] * r.cost;
            if (r.first >= r.seq_first + units) {
                r.seq_first += units;
                continue;
            }
        }
        AttnSeq q;
        bool bad;
        const int mine = attn_seq<M>(p, r.lg, s0 + lane, s0 + lane < attn_seqs<M>(p), &q, &bad)
                             ? attn_units<M>(p, q, RT, r.cost) : 0;
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
    int skip;         // kAttnOwn: pages of the table before page 0; kAttnPrefix: number of the group
};

// The next segment of a CTA's stretch, which starts at unit *at of sequence
// w->seq or a later one; *at moves past it.  False: there is none.  Called by one whole warp.
template <int M>
__device__ __forceinline__ bool attn_next(const AttnParams& p, int RT, AttnRange* w, int* at, AttnSegment* g)
{
    for (int u = *at; u < w->last;) {
        AttnSeq q;
        bool bad;
        const int units = attn_seq<M>(p, w->lg, w->seq, true, &q, &bad) ? attn_units<M>(p, q, RT, w->cost) : 0;
        if (u >= w->seq_first + units) {
            w->seq_first += units;
            if (++w->seq >= attn_seqs<M>(p)) return false;  // not reached unless the lengths change under the call
            continue;
        }
        const int blocks = (q.T * p.group + RT - 1) / RT;
        int g0, end, unit = 1, head, block;  // the group's first unit, its end, units of a page
        if constexpr (M == kAttnPrefix) {
            const int of_head = units / p.c.n_kv_heads, span = p.sh.full * q.pages + w->cost, in = u - w->seq_first;
            head = in / of_head;
            block = min((in - head * of_head) / span, blocks - 1);
            unit = attn_unit(p, q, block);
            g0 = w->seq_first + head * of_head + block * span;
            end = g0 + unit * q.pages + w->cost;
        } else {
            const int span = q.pages + w->cost;
            const int k = u - w->seq_first < span ? 0 : (u - w->seq_first) / span;  // group within the sequence
            g0 = w->seq_first + k * span;
            end = g0 + span;
            head = blocks == 1 ? k : k / blocks;
            block = k - head * blocks;
        }
        const int g1 = g0 + unit * q.pages;
        // a page is the CTA's that has its first unit
        int from = u - g0, to = min(g1, w->last) - g0;
        if constexpr (M == kAttnPrefix) from = (from + unit - 1) / unit, to = (to + unit - 1) / unit;
        if (u >= g1 || from >= to) {
            u = w->last >= g1 ? end : w->last;
            continue;
        }
        g->seq = q.row;
        g->skip = M == kAttnPrefix ? w->seq : q.skip;
        g->t0 = q.t0, g->T = q.T, g->ctx = q.ctx;
        g->head = head;
        g->row0 = block * RT;
        g->page0 = from;
        g->n = to - from;
        const bool whole = from == 0 && to == q.pages;
        g->cta0 = whole ? int(blockIdx.x) : w->owner(g0);
        g->n_ctas = whole ? 1 : w->owner(g1 - unit) - g->cta0 + 1;
        g->slot0 = g0 > w->begin(g->cta0) ? 1 : 0;
        g->slot = u > w->first ? 1 : 0;
        *at = min(g0 + unit * to, w->last);
        return true;
    }
    return false;
}

// a segment's page numbers; its keys' end
template <int M>
__device__ __forceinline__ const int32_t* attn_table(const AttnParams& p, const AttnSegment& g)
{
    return p.c.table + int64_t(g.seq) * p.c.table_ld + g.page0 + (M == kAttnOwn ? g.skip : 0);
}
template <int M>
__device__ __forceinline__ int attn_len(const AttnSegment& g)
{
    return M == kAttnPrefix ? g.ctx : g.ctx + g.T;
}
// whether the segment's rows are left for the join of a prefix and what is behind it
template <int M>
__device__ __forceinline__ bool attn_raw(const AttnSegment& g)
{
    return M == kAttnPrefix || (M == kAttnOwn && g.skip > 0);
}
template <int M>
__device__ __forceinline__ const AttnRows& attn_rows_of(const AttnParams& p)
{
    return M == kAttnPrefix ? p.sh.prefix : p.sh.own;
}
// a query row's place among the rows of a call
__device__ __forceinline__ int64_t attn_place(const AttnParams& p, const AttnSegment& g, int row)
{
    const int node = attn_row_token(p, row);
    return int64_t(g.t0 + node) * p.a.n_heads + (g.head - node) * p.group + row;
}
// where the join finds the row block at row0 of group k, whose tokens start at t0: the blocks of a group have numbers
// of their own, whatever the groups' sizes are
__device__ __forceinline__ int64_t attn_block(const AttnParams& p, int k, int t0, int row0, int head)
{
    return (int64_t(t0) * p.group / kPrefixRows + k + row0 / kPrefixRows) * p.c.n_kv_heads + head;
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
    s[1] = make_int4(g.n_ctas, g.slot0, g.skip, 0);
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

// a row's maximum (less the kernel's shift) and sum, and four of its unnormalised outputs, left for the join
template <int M>
__device__ __forceinline__ void attn_leave_ml(const AttnParams& p, const AttnSegment& g, int row, float m, float l)
{
    attn_rows_of<M>(p).ml[attn_place(p, g, row)] = make_float2(m, l);
}
template <int M>
__device__ __forceinline__ void attn_leave4(const AttnParams& p, const AttnSegment& g, int row, bool there, int D, int d,
                                            float4 v)
{
    if (there) *reinterpret_cast<float4*>(attn_rows_of<M>(p).o + attn_place(p, g, row) * D + d) = v;
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

// a kernel that may start before the one that has just been launched ends
template <class K>
cudaError_t attn_launch_pdl(K kernel, dim3 grid, int threads, size_t smem, const AttnParams& p, unsigned* status,
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
// calls with shared prefixes: the sequences' own keys by the kernels for few and for many rows, the prefixes, the join
cudaError_t launch_attn_own_rows(const mq_kv_cache& cache, const AttnParams& p, int RT, int grid, unsigned* status,
                                 cudaStream_t s);
cudaError_t launch_attn_own_tc(const mq_kv_cache& cache, const AttnParams& p, int grid, unsigned* status, cudaStream_t s);
// the own keys' joins, where they are kernels: behind the prefixes' kernel, which shares the SMs with the first
cudaError_t launch_attn_own_rows_join(const mq_kv_cache& cache, const AttnParams& p, int RT, int grid, unsigned* status,
                                      cudaStream_t s);
cudaError_t launch_attn_own_tc_join(const mq_kv_cache& cache, const AttnParams& p, int grid, unsigned* status,
                                    cudaStream_t s);
cudaError_t launch_attn_shared_join(const mq_kv_cache& cache, const AttnParams& p, unsigned* status, cudaStream_t s);
cudaError_t launch_attn_prefix(const mq_kv_cache& cache, const AttnParams& p, int grid, unsigned* status, cudaStream_t s);
cudaError_t set_attn_own_rows_attributes();
cudaError_t set_attn_own_tc_attributes();
cudaError_t set_attn_prefix_attributes();

// what every attention call puts into its parameters, and where the parts of a workspace lie (attn.cu)
AttnParams attn_params(const mq_kv_cache& cache, const mq_attn_args& a, void* ws, int num_sms);
size_t attn_words_offset(int num_sms);
size_t attn_parts_offset(int num_sms);
int attn_rows_for(int rows);  // query rows of a block of the kernel that takes `rows` per key/value head

}  // namespace mq
