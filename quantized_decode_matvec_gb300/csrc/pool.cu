// pool.cu -- the pages of a key/value cache as a pool: reference counts, a
// stack of free pages, the pages of every sequence (mq_kv_grow, mq_kv_fork,
// mq_kv_free, mq_kv_compact).
//
// Every call does what its list says in the list's order: which page a sequence
// gets, and where a freed one lies on the stack, follows from prefix sums over
// the list, never from the order in which threads come.  The sums are one CTA's
// work, or one cluster's where all references of the call, or all pages of the
// pool, have to be looked at; bytes are then copied by a kernel behind it, on all
// SMs.  Bound by the copied bytes in large calls, by the chain of launches,
// barriers and dependent loads (page table, count, stack) in small ones: a fork of
// 128 sequences of 500 to 9000 tokens (f16, 36 MB copied) 12.3 us, of 3 6.3; growing 64
// sequences by a page 3.2, where none needs one 2.3, 512 by 20 pages 17 (the counts'
// atomics of one SM); free of 16 sequences 7; a compaction of 4923 pages that moves
// 142 MB 33, of which the moves are 22 (6.5 TB/s).
// Nothing on the device is trusted: an entry that contradicts the pool is left
// out, and sets MQ_DEV_KV_RANGE.  The counts are what the calls go by: a page is free
// at 0, in use above, and nothing is handed out, shared or pushed against that.  (A
// fork of 3 took 5.5 us and of 128 10.7 without the checks.)
#include <cooperative_groups.h>

#include "mq_internal.h"
#include "mq_kv.cuh"
#include "mq_stream.cuh"

namespace mq {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kSeqs = MQ_MAX_SEQS, kPer = kSeqs / kThreads;  // entries of a thread
constexpr int kCluster = 8;
constexpr int kSkip = -2, kNone = -1;  // an entry left out; one that needs no page

struct PoolArgs {
    KvView c;
    int32_t* table;
    mq_kv_pool pool;
    const int32_t* a;  // grow: lengths; fork: sources; free: sequences
    const int32_t* b;  // fork: new sequences; free: pages kept, or null
    const int32_t* len;  // fork
    int n;
    int page_bytes;
};

// exclusive prefix sums over the CTA of kPer consecutive values per thread; returns the total
__device__ __forceinline__ int scan(const int (&v)[kPer], int (&out)[kPer], int* warp_s)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum += v[k];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += w;
    }
    __syncthreads();  // the words of the scan before are read
    if (lane == 31) warp_s[warp] = incl;
    __syncthreads();
    int w = warp_s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    const int total = __shfl_sync(0xffffffffu, w, 31), base = __shfl_sync(0xffffffffu, w, warp) - warp_s[warp];
    int at = base + incl - sum;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        out[k] = at;
        at += v[k];
    }
    return total;
}

// the last entry whose first position is not past pos (off_s[0] = 0, n + 1 of them)
__device__ __forceinline__ int entry_of(const int* off_s, int n, int pos)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (off_s[mid] <= pos)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// n: *p.pool.n_free, which is loaded ahead of the sums
__device__ __forceinline__ int free_pages(const PoolArgs& p, int n, bool* bad)
{
    *bad = n < 0 || n > p.c.n_pages;
    return *bad ? 0 : n;
}

// Takes a free page: false where the stack names none (a page outside the pool, or one with a count: in use, or named
// twice).  The count becomes 1; give_back undoes that.
__device__ __forceinline__ bool take_page(const PoolArgs& p, int page)
{
    return page >= 0 && page < p.c.n_pages && atomicCAS(p.pool.refs + page, 0, 1) == 0;
}
__device__ __forceinline__ void give_back(const PoolArgs& p, int page) { p.pool.refs[page] = 0; }

// ---- grow -----------------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) grow_kernel(const PoolArgs p, unsigned* status)
{
    __shared__ int off_s[kSeqs + 1], have_s[kSeqs], warp_s[kWarps];
    const int tid = threadIdx.x, n = p.c.n_seqs, stack = __ldcg(p.pool.n_free);
    int v[kPer], at[kPer];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int s = tid * kPer + k;
        v[k] = 0;
        if (s >= n) continue;
        const int have = p.pool.seq_pages[s], len = __ldg(p.a + s);
        const int64_t want = (int64_t(len) + kKvPage - 1) / kKvPage;
        have_s[s] = have;
        if (have < 0 || have > p.c.table_ld || len < 0 || want > p.c.table_ld)
            bad = true;
        else if (want > have)
            v[k] = int(want) - have;
    }
    const int total = scan(v, at, warp_s);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (tid * kPer + k < n) off_s[tid * kPer + k] = at[k];
    if (tid == 0) off_s[n] = total;
    bool bad_free;
    const int n_free = free_pages(p, stack, &bad_free);
    if (__syncthreads_or(bad) || bad_free) {
        if (tid == 0) atomicOr(status, MQ_DEV_KV_RANGE);
    }
    if (total == 0) return;
    if (total > n_free) {
        if (tid == 0) atomicOr(status, MQ_DEV_KV_FULL);
        return;
    }
    // all pages are taken before any is written down: where the stack names one that is not free, none is
    int got = 0;  // the thread's, up to the first that is not
    while (tid + got * kThreads < total && take_page(p, p.pool.free_list[n_free - 1 - tid - got * kThreads])) ++got;
    if (__syncthreads_or(tid + got * kThreads < total)) {
        if (tid == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        for (int k = 0; k < got; ++k) give_back(p, p.pool.free_list[n_free - 1 - tid - k * kThreads]);
        return;
    }
    for (int pos = tid; pos < total; pos += kThreads) {
        const int s = entry_of(off_s, n, pos);
        p.table[int64_t(s) * p.c.table_ld + have_s[s] + pos - off_s[s]] = p.pool.free_list[n_free - 1 - pos];
    }
    for (int s = tid; s < n; s += kThreads)
        if (off_s[s + 1] > off_s[s]) p.pool.seq_pages[s] = have_s[s] + off_s[s + 1] - off_s[s];
    if (tid == 0) *p.pool.n_free = n_free - total;
}

// ---- fork -----------------------------------------------------------------------------------
// The plan: for every entry the page that it takes for its begun page, kNone or kSkip, in the scratch.
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const PoolArgs p, unsigned* status)
{
    __shared__ int warp_s[kWarps];
    __shared__ int dst_s[kSeqs];          // the first entry that forks into a sequence
    __shared__ uint32_t src_s[kSeqs / 32];  // sequences that an entry forks from
    griddep_launch_dependents();
    const int tid = threadIdx.x, stack = __ldcg(p.pool.n_free);
    for (int i = tid; i < kSeqs; i += kThreads) dst_s[i] = INT32_MAX;
    if (tid < kSeqs / 32) src_s[tid] = 0;
    __syncthreads();
    int src[kPer], dst[kPer], len[kPer];
    bool ok[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        ok[k] = false;
        if (i >= p.n) continue;
        src[k] = __ldg(p.a + i), dst[k] = __ldg(p.b + i), len[k] = __ldg(p.len + i);
        const bool in = src[k] >= 0 && src[k] < p.c.n_seqs && dst[k] >= 0 && dst[k] < p.c.n_seqs && len[k] >= 0;
        if (in) {
            const int pages = p.pool.seq_pages[src[k]];
            ok[k] = pages >= 0 && pages <= p.c.table_ld && (int64_t(len[k]) + kKvPage - 1) / kKvPage <= pages &&
                    p.pool.seq_pages[dst[k]] == 0;
            atomicMin(&dst_s[dst[k]], i);
            atomicOr(&src_s[src[k] / 32], 1u << src[k] % 32);
        }
    }
    __syncthreads();
    int v[kPer], at[kPer];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        // a new sequence is named once, and nothing is forked from it in the same call
        ok[k] = ok[k] && dst_s[dst[k]] == i && !(src_s[dst[k] / 32] >> dst[k] % 32 & 1);
        bad |= i < p.n && !ok[k];
        v[k] = ok[k] && len[k] % kKvPage ? 1 : 0;
    }
    const int total = scan(v, at, warp_s);
    bool bad_free;
    const int n_free = free_pages(p, stack, &bad_free);
    if (__syncthreads_or(bad) || bad_free) {
        if (tid == 0) atomicOr(status, MQ_DEV_KV_RANGE);
    }
    const bool full = total > n_free;
    if (full && tid == 0) atomicOr(status, MQ_DEV_KV_FULL);
    int page[kPer];
    bool wrong = false, took[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        page[k] = ok[k] && !full ? kNone : kSkip;
        took[k] = false;
        if (page[k] == kNone && v[k]) {
            page[k] = p.pool.free_list[n_free - 1 - at[k]];
            took[k] = take_page(p, page[k]);
            wrong |= !took[k];
        }
    }
    wrong = __syncthreads_or(wrong);  // the stack names a page that is not free: nothing is forked
    if (wrong && tid == 0) atomicOr(status, MQ_DEV_KV_RANGE);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        if (wrong && took[k]) give_back(p, page[k]);
        if (i < p.n) p.pool.scratch[i] = wrong ? kSkip : page[k];
    }
    if (tid == 0 && !full && !wrong && total) *p.pool.n_free = n_free - total;
}

// by `step` threads, number `at` of which calls; their first kAhead loads are on their way together
template <int kAhead>
__device__ __forceinline__ void copy16(uint8_t* dst, const uint8_t* src, int bytes, int at, int step)
{
    const int n = bytes / 16;
    for (int i = at; i < n; i += kAhead * step) {
        uint4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * step < n) v[k] = __ldg(reinterpret_cast<const uint4*>(src) + i + k * step);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * step < n) reinterpret_cast<uint4*>(dst)[i + k * step] = v[k];
    }
}

// CTA (entry, key/value head): the begun page's written rows of the head; head 0's also the table and the counts
template <int D, bool Q8>
__global__ void __launch_bounds__(256) fork_copy_kernel(const PoolArgs p, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    const int e = blockIdx.x, h = blockIdx.y;
    const int src = __ldg(p.a + e), dst = __ldg(p.b + e), len = __ldg(p.len + e);
    const int full = len / kKvPage, rest = len % kKvPage;
    const int32_t* const from = p.table + int64_t(src) * p.c.table_ld;
    int32_t* const to = p.table + int64_t(dst) * p.c.table_ld;
    // the source's pages, which the plan leaves as they are, ahead of it: a thread's first, and the begun one
    const bool known = src >= 0 && src < p.c.n_seqs && len >= 0;
    const int first = known && h == 0 && threadIdx.x < min(full, p.c.table_ld) ? __ldcg(from + threadIdx.x) : -1;
    const int begun = known && full < p.c.table_ld ? __ldcg(from + full) : -1;
    griddep_wait();
    const int page = __ldcg(p.pool.scratch + e);
    if (page == kSkip) return;
    if (h == 0) {
        for (int i = threadIdx.x; i < full; i += 256) {
            // a page that nobody has is on the stack, or lost: it is not shared (no other entry makes it one with a
            // count, since none takes such a one)
            int x = i < 256 ? first : from[i];
            if (x < 0 || x >= p.c.n_pages || __ldcg(p.pool.refs + x) <= 0) x = -1;
            to[i] = x;
            if (x >= 0)
                atomicAdd(p.pool.refs + x, 1);
            else
                atomicOr(status, MQ_DEV_KV_RANGE);
        }
        if (threadIdx.x == 0) {
            if (rest) to[full] = page;
            p.pool.seq_pages[dst] = full + (rest != 0);
        }
    }
    if (rest == 0) return;
    const int x = begun;
    if (x < 0 || x >= p.c.n_pages) {  // nothing to copy: the new page stays as it was
        if (threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    const uint8_t* const in = p.c.pages + (int64_t(x) * p.c.n_kv_heads + h) * B::kBytes;
    uint8_t* const out = p.c.pages + (int64_t(page) * p.c.n_kv_heads + h) * B::kBytes;
    // K's and V's planes by a share of the threads each, every byte of a thread in one round
    constexpr int kPlanes = 2 * (Q8 ? 1 : D / 64), kShare = 256 / kPlanes;
    const int k = threadIdx.x / kShare;
    copy16<kKvPage * B::kRow / 16 / kShare>(out + k * kKvPage * B::kRow, in + k * kKvPage * B::kRow, rest * B::kRow,
                                            threadIdx.x % kShare, kShare);
    if (Q8) {
        constexpr int kWords = D / 64;  // 32-bit words of a row's scales
        for (int i = threadIdx.x; i < 2 * rest * kWords; i += 256) {
            const int at = B::kScK + (i >= rest * kWords ? B::kScBytes - rest * kWords * 4 : 0) + i * 4;
            *reinterpret_cast<uint32_t*>(out + at) = __ldg(reinterpret_cast<const uint32_t*>(in + at));
        }
    }
}

// ---- a cluster's view of a call -------------------------------------------------------------
struct ClusterSum {
    int warp[kWarps];
    int2 total[4];  // sum and flag, by use; read by the whole cluster
};

// Sum of v over the CTA, all CTAs' sums met: *before those of the CTAs before this one; returns the cluster's.  *any:
// whether one thread's flag was set.  Global writes before it are seen by the cluster behind it (the barrier releases
// and acquires).
__device__ __forceinline__ int cluster_sum(cg::cluster_group& cl, ClusterSum& s, int use, int v, int* before, bool flag = false,
                                           int* any = nullptr)
{
    v = __reduce_add_sync(0xffffffffu, v);
    flag = __syncthreads_or(flag);
    if (threadIdx.x % 32 == 0) s.warp[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int all = __reduce_add_sync(0xffffffffu, s.warp[threadIdx.x]);
        if (threadIdx.x == 0) s.total[use] = make_int2(all, flag);
    }
    cl.sync();
    // a lane per CTA: one after the other these loads take 0.3 us each
    const int c = threadIdx.x % 32;
    const int2 w = c < int(cl.num_blocks()) ? *cl.map_shared_rank(&s.total[use], c) : make_int2(0, 0);
    const int all = __reduce_add_sync(0xffffffffu, w.x), flags = __any_sync(0xffffffffu, w.y != 0);
    *before = __reduce_add_sync(0xffffffffu, c < int(cl.block_rank()) ? w.x : 0);
    if (any) *any = flags;
    return all;
}

// rank of a thread's flag among the CTA's, and how many there are
__device__ __forceinline__ int cta_rank(bool flag, int* warp_s, int* count)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const unsigned b = __ballot_sync(0xffffffffu, flag);
    __syncthreads();
    if (lane == 0) warp_s[warp] = __popc(b);
    __syncthreads();
    int w = warp_s[lane];
    const int mine = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    *count = __shfl_sync(0xffffffffu, w, 31);
    return __shfl_sync(0xffffffffu, w - mine, warp) + __popc(b & ((1u << lane) - 1));
}

// ---- free -----------------------------------------------------------------------------------
// Positions are the references that the call gives up, in its order.  A page whose count comes to zero is pushed at
// its last position.  A page without a count, or that the call names more often than its count says, contradicts the
// pool: the first stays as it is, the second is pushed once.  scratch[page]: the page's last position in the call;
// scratch[n_pages + page]: how often the call names it (both only where a page may be named twice).
__global__ void __launch_bounds__(kThreads) free_kernel(const PoolArgs p, unsigned* status)
{
    __shared__ int off_s[kSeqs + 1], warp_s[kWarps];
    __shared__ int first_s[kSeqs];  // by sequence: the first entry that names it
    __shared__ ClusterSum sum_s;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, rank = int(cl.block_rank()), stack = __ldcg(p.pool.n_free);
    for (int i = tid; i < kSeqs; i += kThreads) first_s[i] = INT32_MAX;
    __syncthreads();
    int seq[kPer], keep[kPer], have[kPer], v[kPer], at[kPer];
    bool bad = false, ok[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        ok[k] = false, v[k] = 0, seq[k] = 0, keep[k] = 0, have[k] = 0;
        if (i >= p.n) continue;
        seq[k] = __ldg(p.a + i), keep[k] = p.b ? __ldg(p.b + i) : 0;
        ok[k] = seq[k] >= 0 && seq[k] < p.c.n_seqs && keep[k] >= 0;
        if (ok[k]) {
            have[k] = __ldcg(p.pool.seq_pages + seq[k]);
            ok[k] = have[k] >= 0 && have[k] <= p.c.table_ld;
            atomicMin(&first_s[seq[k]], i);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        if (i >= p.n) continue;
        ok[k] = ok[k] && first_s[seq[k]] == i;
        bad |= !ok[k];
        v[k] = ok[k] && have[k] > keep[k] ? have[k] - keep[k] : 0;
    }
    const int total = scan(v, at, warp_s);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (tid * kPer + k < p.n) off_s[tid * kPer + k] = at[k];
    if (tid == 0) off_s[p.n] = total;
    bool bad_free;
    const int n_free = free_pages(p, stack, &bad_free);
    if (__syncthreads_or(bad) || bad_free) {
        if (tid == 0 && rank == 0) atomicOr(status, MQ_DEV_KV_RANGE);
    }
    if (total == 0 || bad_free) return;  // the same in the whole cluster
    const int ctas = int(cl.num_blocks());
    const int per = (total + ctas - 1) / ctas, begin = min(rank * per, total), end = min(begin + per, total);
    // the table's entry at a position; its page, or -1
    auto place = [&](int pos, int64_t* where) {
        const int e = entry_of(off_s, p.n, pos), s = __ldg(p.a + e), k = p.b ? __ldg(p.b + e) : 0;
        *where = int64_t(s) * p.c.table_ld + k + pos - off_s[e];
        const int page = __ldcg(p.table + *where);
        return page >= 0 && page < p.c.n_pages ? page : -1;
    };
    // a page with one reference goes where that is; only of one that others name too has the last to be found, which is
    // any whose count was not one
    int32_t* const last = p.pool.scratch;
    int32_t* const named = p.pool.scratch + p.c.n_pages;
    int64_t w;
    int page, before, alone = 0, shared = 0;
    int page0 = -1;  // of the thread's first position, which is its only one mostly: kept, with the rest of it
    int64_t w0 = 0;
    for (int pos = begin + tid; pos < end; pos += kThreads) {
        page = place(pos, &w);
        if (pos == begin + tid) page0 = page, w0 = w;
        if (page < 0) {
            atomicOr(status, MQ_DEV_KV_RANGE);
            continue;
        }
        const int refs = atomicSub(p.pool.refs + page, 1);
        alone += refs == 1;
        shared |= refs != 1;
        __stcg(last + page, -1);
        __stcg(named + page, 0);
    }
    int pushed = cluster_sum(cl, sum_s, 0, alone, &before, shared, &shared);
    // whether a position is where its page is pushed; *count: the page's count before the call, less what the call names
    auto freed = [&](int pos, int* page, int64_t* where, int* count) {
        *page = place(pos, where);
        *count = 0;
        if (*page < 0) return false;
        if (!shared) return true;
        if (__ldcg(last + *page) != pos) return false;
        *count = __ldcg(p.pool.refs + *page);
        return *count <= 0 && *count + __ldcg(named + *page) > 0;
    };
    int rest;
    if (shared) {  // the same in the whole cluster
        for (int pos = begin + tid; pos < end; pos += kThreads) {
            if ((page = place(pos, &w)) >= 0) {
                atomicMax(last + page, pos);
                atomicAdd(named + page, 1);
            }
        }
        cl.sync();
        int count = 0;
        for (int pos = begin + tid; pos < end; pos += kThreads) {
            count += freed(pos, &page, &w, &rest);
            if (rest < 0) atomicOr(status, MQ_DEV_KV_RANGE);
        }
        pushed = cluster_sum(cl, sum_s, 1, count, &before);
    }
    if (n_free + pushed > p.c.n_pages) {  // the stack names pages that are in use
        if (tid == 0 && rank == 0) atomicOr(status, MQ_DEV_KV_RANGE);
    }
    for (int base = begin; base < end; base += kThreads) {
        const int pos = base + tid;
        bool flag = false;
        rest = 0;
        if (base == begin && !shared) {
            flag = pos < end && page0 >= 0;
            page = page0, w = w0;
        } else if (pos < end) {
            flag = freed(pos, &page, &w, &rest);
        }
        int here;
        const int to = n_free + before + cta_rank(flag, warp_s, &here);
        if (flag && to < p.c.n_pages) p.pool.free_list[to] = page;
        // below zero: named too often, or without a count before, which it has again
        if (rest < 0) p.pool.refs[page] = flag ? 0 : rest + __ldcg(named + page);
        if (pos < end) p.table[w] = -1;
        before += here;
    }
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (ok[k] && have[k] > keep[k]) p.pool.seq_pages[seq[k]] = keep[k];
        if (tid == 0) *p.pool.n_free = int(min(int64_t(n_free) + pushed, p.c.n_pages));
    }
    cl.sync();
}

// ---- compact --------------------------------------------------------------------------------
// With U pages in use, the k-th page in use from U on goes to the k-th free one before U.  scratch: n_pages words,
// the place that a page in use goes to, -1 of one that is not; then the free pages before U in ascending order, and the pages in use from
// U on in descending order (their ranks among all pages in use are known before their number is); then both's number.
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const PoolArgs p, unsigned* status)
{
    __shared__ int warp_s[kWarps];
    __shared__ ClusterSum sum_s;
    griddep_launch_dependents();
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, rank = int(cl.block_rank()), ctas = int(cl.num_blocks()), n = int(p.c.n_pages);
    const int per = (n + ctas - 1) / ctas;
    const int begin = int(min(int64_t(rank) * per, int64_t(n))), end = int(min(int64_t(begin) + per, int64_t(n)));
    int32_t* const map = p.pool.scratch;
    int32_t* const hole = map + n;
    int32_t* const far = hole + (n + 1) / 2;
    int count = 0, before;
    for (int i = begin + tid; i < end; i += kThreads) count += p.pool.refs[i] > 0;
    const int used = cluster_sum(cl, sum_s, 0, count, &before);
    int holes = 0, unused;
    for (int base = begin; base < end; base += kThreads) {
        const int i = base + tid;
        const int refs = i < end ? p.pool.refs[i] : 0;
        const bool in_use = refs > 0;
        int here;
        const int at = before + cta_rank(in_use, warp_s, &here);  // pages in use before page i
        if (refs < 0) {
            p.pool.refs[i] = 0;
            atomicOr(status, MQ_DEV_KV_RANGE);
        }
        if (i < end && !(i >= used && in_use)) __stcg(map + i, in_use ? i : -1);
        if (i < end && i < used && !in_use) __stcg(hole + i - at, i), ++holes;
        if (i >= used && in_use) __stcg(far + used - 1 - at, i);
        if (i >= used && i < end) p.pool.free_list[n - 1 - i] = i;
        before += here;
    }
    const int moves = cluster_sum(cl, sum_s, 1, holes, &unused);
    for (int k = rank * kThreads + tid; k < moves; k += ctas * kThreads) {
        const int from = __ldcg(far + moves - 1 - k), to = __ldcg(hole + k);
        map[from] = to;
        p.pool.refs[to] = p.pool.refs[from];
        p.pool.refs[from] = 0;
    }
    if (rank == 0 && tid == 0) {
        *p.pool.n_free = n - used;
        map[2 * n + 2] = moves;
    }
    cl.sync();
}

constexpr int kMoveThreads = 256, kMoveBytes = 16 * 1024;  // of a CTA's turn

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const PoolArgs p, unsigned* status)
{
    griddep_wait();
    const int n = int(p.c.n_pages), moves = __ldcg(p.pool.scratch + 2 * n + 2);
    const int32_t* const hole = p.pool.scratch + n;
    const int32_t* const far = hole + (n + 1) / 2;
    const int parts = (p.page_bytes + kMoveBytes - 1) / kMoveBytes;
    for (int64_t w = blockIdx.x; w < int64_t(moves) * parts; w += gridDim.x) {
        const int k = int(w / parts), at = int(w % parts) * kMoveBytes;
        copy16<4>(p.c.pages + int64_t(__ldcg(hole + k)) * p.page_bytes + at,
                  p.c.pages + int64_t(__ldcg(far + moves - 1 - k)) * p.page_bytes + at, min(kMoveBytes, p.page_bytes - at),
                  threadIdx.x, kMoveThreads);
    }
    for (int64_t i = int64_t(blockIdx.x) * kMoveThreads + threadIdx.x; i < int64_t(p.c.n_seqs) * p.c.table_ld;
         i += int64_t(gridDim.x) * kMoveThreads) {
        const int s = int(i / p.c.table_ld), have = p.pool.seq_pages[s], at = int(i - int64_t(s) * p.c.table_ld);
        if (at == 0 && (have < 0 || have > p.c.table_ld)) atomicOr(status, MQ_DEV_KV_RANGE);
        if (at >= have) continue;
        // an entry that names a page that is not in use names none from now on: another one's may come to lie there
        const int page = p.table[i], to = page >= 0 && page < n ? __ldcg(p.pool.scratch + page) : -1;
        if (to < 0) atomicOr(status, MQ_DEV_KV_RANGE);
        if (to != page) p.table[i] = to;
    }
}

// One CTA where its threads have an item each, else a cluster.  The plan of 4923 pages 7 us; in an earlier form 10, and
// 15 by one CTA.
template <class K, class... A>
cudaError_t launch_cluster(K kernel, int64_t items, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    const int ctas = items <= kThreads ? 1 : kCluster;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class K>
cudaError_t launch_behind(K kernel, dim3 grid, int threads, cudaStream_t s, const PoolArgs& p, unsigned* status)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, status);
}

PoolArgs pool_args(const mq_kv_cache& c, const mq_kv_pool& pool)
{
    PoolArgs p = {};
    p.c = kv_view(c);
    p.table = const_cast<int32_t*>(c.table);
    p.pool = pool;
    p.page_bytes = int(mq_kv_page_bytes(c.type, c.n_kv_heads, c.head_dim));
    return p;
}

}  // namespace

cudaError_t launch_kv_grow(const mq_kv_cache& c, const mq_kv_pool& pool, const int32_t* length, unsigned* status,
                           cudaStream_t s)
{
    PoolArgs p = pool_args(c, pool);
    p.a = length;
    grow_kernel<<<1, kThreads, 0, s>>>(p, status);
    return cudaGetLastError();
}

cudaError_t launch_kv_fork(const mq_kv_cache& c, const mq_kv_pool& pool, const int32_t* src, const int32_t* dst,
                           const int32_t* length, int n, unsigned* status, cudaStream_t s)
{
    PoolArgs p = pool_args(c, pool);
    p.a = src, p.b = dst, p.len = length, p.n = n;
    fork_plan_kernel<<<1, kThreads, 0, s>>>(p, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const dim3 grid(n, c.n_kv_heads);
    if (c.type == MQ_TYPE_Q8_0)
        return c.head_dim == 128 ? launch_behind(fork_copy_kernel<128, true>, grid, 256, s, p, status)
                                 : launch_behind(fork_copy_kernel<64, true>, grid, 256, s, p, status);
    return c.head_dim == 128 ? launch_behind(fork_copy_kernel<128, false>, grid, 256, s, p, status)
                             : launch_behind(fork_copy_kernel<64, false>, grid, 256, s, p, status);
}

cudaError_t launch_kv_free(const mq_kv_cache& c, const mq_kv_pool& pool, const int32_t* seq, const int32_t* keep, int n,
                           unsigned* status, cudaStream_t s)
{
    PoolArgs p = pool_args(c, pool);
    p.a = seq, p.b = keep, p.n = n;
    return launch_cluster(free_kernel, int64_t(n) * c.table_ld, s, p, status);
}

cudaError_t launch_kv_compact(const mq_kv_cache& c, const mq_kv_pool& pool, int num_sms, unsigned* status, cudaStream_t s)
{
    PoolArgs p = pool_args(c, pool);
    const cudaError_t e = launch_cluster(compact_plan_kernel, c.n_pages, s, p, status);
    if (e != cudaSuccess) return e;
    return launch_behind(compact_move_kernel, dim3(unsigned(num_sms) * 8), kMoveThreads, s, p, status);
}

}  // namespace mq
