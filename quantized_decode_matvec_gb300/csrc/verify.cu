// verify.cu -- verification of drafted trees against the target's
// probabilities, from given random numbers (mq_verify_tree).
//
// At a node with target row p and draft row q, children x_1, x_2, .. (drawn from
// q) are tried in order against what the refused ones have left of p:
//   S_k = (p - a_k q)+,  W_k = sum S_k,   a_0 = 0, W_0 = 1,   a_(k+1) = a_k + W_k
// (the residual (R_k - q)+ of the normalised R_k = S_k / W_k, scaled by W_k).
// Child x is accepted where u q(x) W_k < S_k(x); the walk goes on at the first
// that is.  Where none is, the last S is what the next token is drawn from: the
// first index at which the running sum of S passes u W.
//
// Which token comes out hangs on sums over a vocabulary, so probabilities are
// rounded to multiples of 2^-46 and summed as integers, so that no sum depends on
// its order; over 2^17 values the roundings come to some 2^-39, and the chance that
// they change a draw is about 3e-7 (a sum in fp32 would change one in 70).  Two
// 23-bit halves per value, in 32-bit arithmetic: with 64-bit numbers in units of
// 2^-60 the pass was bound by some 45 instructions per value.  A test of a child is
// one comparison in 64-bit floating point.
//
// A cluster of CTAs per sequence: each takes a contiguous part of the
// vocabulary, and keeps the sums of its tiles, so that the draw looks into one
// tile only.  Every CTA walks the tree by itself from the same numbers; they meet
// where a row's sum is needed, which is once for every refused child, and once
// more at a node without children.  Bound by the chain of loads, passes and
// barriers: 131072 values, children refused at the root 0, 1, 2 and 3: one sequence
// 8.4, 12.4, 18 and 25 us, 64 of them 13.7, 22, 38 and 53 (a pass reads 67 MB then);
// 64 trees of 16 nodes 47 us, greedy, with 2.8 passes each, 74.  64 registers, the
// most that four CTAs per SM leave, spill 40 bytes.
#include <cooperative_groups.h>

#include "mq_internal.h"
#include "mq_tma.cuh"

namespace mq {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxNodes = MQ_TREE_MAX_TOKENS;
constexpr int kMaxCluster = 16;
constexpr int kUnit = 512;       // values of a warp's step: 16 per lane
constexpr int kMaxTiles = 1024;  // of a CTA
constexpr int kHalf = 23, kOne = 2 * kHalf;  // 1.0 is 2^46
constexpr double kInvOne = 1.0 / double(1ull << kOne);
// A row that sums to 2^17 or more holds no probabilities.  Up to 2^18 values of at most 1 their sums stay in range as
// unsigned numbers; of more they stop at this one.  (A warp's part of a tile is below 2^62: kMaxTiles tiles hold 2^28 / 8
// values.)
constexpr uint64_t kTooMuch = (1ull << 63) - 1;

struct VerifyArgs {
    mq_verify_args a;
    bool capped;      // sums may pass 64 bits
    int chunk, tile;  // places of a CTA (a multiple of tile) and of a tile (a multiple of kUnit)
};

// A probability in units of 2^-46, rounded to nearest: hi 2^23 + lo.  What is not a number above zero is zero, what is
// above one is one.  Adding 1 leaves the first 23 bits in the mantissa, what they leave is exact, and so are its next 23.
struct Fixed {
    int hi, lo;
};
__device__ __forceinline__ Fixed halves(float p)
{
    p = __saturatef(p);
    const float f = __fadd_rz(p, 1.0f), rest = p - (f - 1.0f), g = fmaf(rest, 8388608.0f, 1.0f);
    return Fixed{__float_as_int(f) - 0x3f800000, __float_as_int(g) - 0x3f800000};
}
__device__ __forceinline__ uint64_t whole(int hi, int lo) { return (uint64_t(uint32_t(hi)) << kHalf) + uint32_t(lo); }
__device__ __forceinline__ uint64_t fixed(float p)
{
    const Fixed x = halves(p);
    return whole(x.hi, x.lo);
}

// p - a q where that is above zero, else 0, for a of two parts: the product in two parts, whose second is rounded to the
// unit by itself.  A difference of rounded numbers that comes out below zero is zero.
__device__ __forceinline__ Fixed less(float p, float q, float a_hi, float a_lo)
{
    p = __saturatef(p), q = __saturatef(q);
    const float y = a_hi * q, rest = fmaf(a_lo, q, fmaf(a_hi, q, -y));
    if (!((p - y) - rest > 0.0f)) return Fixed{0, 0};
    const Fixed P = halves(p), Y = halves(y);
    const int hi = P.hi - Y.hi, lo = P.lo - Y.lo - (__float_as_int(fmaf(rest, 0x1p46f, 12582912.0f)) - 0x4b400000);
    return hi <= 1 && hi * (1 << kHalf) + lo < 0 ? Fixed{0, 0} : Fixed{hi, lo};
}

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t warp_sum(uint64_t v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// of numbers up to kTooMuch, as such a one
__device__ __noinline__ uint64_t warp_sum_capped(uint64_t v)
{
    for (int o = 16; o; o >>= 1) v = min(v + __shfl_xor_sync(0xffffffffu, v, o), kTooMuch);
    return v;
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = larger(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

enum { kEnd, kAccept, kRefuse };

struct Shared {
    int tok[kMaxNodes], par[kMaxNodes];
    float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];  // p, q: of the node's token at its parent
    unsigned long long kids[kMaxNodes];              // of every node, a bit each
    int path[kMaxNodes], gone[kMaxNodes];            // gone: refused tokens of the node at hand (point masses)
    uint64_t tile[kMaxTiles];
    uint64_t warp[kWarps];
    uint64_t total[2];  // read by the whole cluster; of every other pass
    int found;
    int act, child;     // what the walk does next
    float a_hi, a_lo;
    int n_gone;
};

// S at one index, in fixed point
struct Residual {
    const float* p;
    const float* q;  // or null
    float a_hi, a_lo;  // 0: the row as it is
    int n_gone;
    const int* gone;
    __device__ __forceinline__ int64_t of(float pv, float qv) const
    {
        if (a_hi == 0.0f) return int64_t(fixed(pv));
        const Fixed x = less(pv, qv, a_hi, a_lo);
        return int64_t(x.hi) * (1 << kHalf) + x.lo;
    }
    __device__ __forceinline__ int64_t at(int i) const
    {
        for (int k = 0; k < n_gone; ++k)
            if (gone[k] == i) return 0;
        return of(__ldg(p + i), a_hi != 0.0f ? __ldg(q + i) : 0.0f);
    }
};

// the order of fp32 numbers as unsigned integers (NaN and -inf: 0)
__device__ __forceinline__ uint32_t ordered(float v)
{
    if (!(v > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(v);
    return b == 0x80000000u ? 0x80000000u : b & 0x80000000u ? ~b : b | 0x80000000u;  // -0 is 0
}

// One pass over the CTA's part of a row: f(index, p, q) of every value, lanes of a warp on neighbouring ones, the
// tiles of the part going round the warps; step() behind every 16 of a lane, done(tile) behind a tile.  Places are counted from the 16-byte boundary before
// the row, `off` values before its first, so that they are read 16 bytes at a time wherever rows start.
template <bool Both, class F, class Step, class Done>
__device__ __forceinline__ void walk_row(const VerifyArgs& p, const float* prow, const float* qrow, int off, int first,
                                         int last, F f, Step step, Done done)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool wide = !Both || (int(reinterpret_cast<uintptr_t>(qrow) >> 2) & 3) == off;
    for (int t = warp; first + t * int64_t(p.tile) < last; t += kWarps) {
        const int begin = first + t * p.tile, end = last - begin < p.tile ? last : begin + p.tile;
        for (int i = begin; i < end; i += kUnit) {
            if (wide && i >= off && end - i >= kUnit) {
                float4 x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = __ldg(reinterpret_cast<const float4*>(prow + (i - off) + j * 128) + lane);
                    if (Both) y[j] = __ldg(reinterpret_cast<const float4*>(qrow + (i - off) + j * 128) + lane);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = i - off + j * 128 + lane * 4;
                    f(k, x[j].x, Both ? y[j].x : 0.0f);
                    f(k + 1, x[j].y, Both ? y[j].y : 0.0f);
                    f(k + 2, x[j].z, Both ? y[j].z : 0.0f);
                    f(k + 3, x[j].w, Both ? y[j].w : 0.0f);
                }
            } else {
#pragma unroll 4
                for (int j = 0; j < kUnit / 32; ++j) {
                    const int k = i - off + j * 32 + lane;
                    if (k >= 0 && k < end - off) f(k, __ldg(prow + k), Both ? __ldg(qrow + k) : 0.0f);
                }
            }
            step();
        }
        done(t);
    }
}

// Four CTAs per SM, so that a batch of 64 sequences is on the chip at once.
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs p, unsigned* status)
{
    __shared__ Shared sm;
    cg::cluster_group cl = cg::this_cluster();
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank()), tid = threadIdx.x;
    const int s = blockIdx.x / C, V = p.a.vocab;
    const bool greedy = (p.a.flags & MQ_VERIFY_GREEDY) != 0;
    const int t0 = __ldg(p.a.tok_start + s);
    const int64_t T64 = int64_t(__ldg(p.a.tok_start + s + 1)) - t0;
    if (t0 < 0 || T64 < 0 || T64 > kMaxNodes || t0 + T64 > p.a.n_tokens) {  // the same in the whole cluster
        if (rank == 0 && tid == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    const int T = int(T64);
    if (T == 0) {
        if (rank == 0 && tid == 0) p.a.n_path[s] = 0, p.a.next[s] = -1;
        for (int i = tid; rank == 0 && i < p.a.path_ld; i += kThreads) p.a.path[int64_t(s) * p.a.path_ld + i] = 0;
        return;
    }
    if (tid < T) {
        const int tok = __ldg(p.a.token + t0 + tid), par = __ldg(p.a.parent + t0 + tid);
        const bool ok = tid > 0 && par >= 0 && par < tid && tok >= 0 && tok < V;
        if (tid > 0 && !ok && rank == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        sm.tok[tid] = tok;
        sm.par[tid] = ok ? par : -1;  // never a child
        sm.kids[tid] = 0;
        if (!greedy) {
            sm.u[tid] = __ldg(p.a.u + t0 + tid);
            // of the numbers that the sums are of, too: NaN and what is below 0 are 0, above 1 is 1
            sm.p[tid] = ok ? __saturatef(__ldg(p.a.target + (t0 + par) * p.a.target_ld + tok)) : 0.0f;
            sm.q[tid] = ok && p.a.draft ? __saturatef(__ldg(p.a.draft + (t0 + par) * p.a.draft_ld + tok)) : 1.0f;
        }
    }
    // the CTA's places in a row that starts `off` values behind a 16-byte boundary
    const int first = int(min(int64_t(rank) * p.chunk, int64_t(V) + 3));
    auto offset = [](const float* row) { return int(reinterpret_cast<uintptr_t>(row) >> 2) & 3; };
    auto end_of = [&](int off) { return int(min(int64_t(first) + p.chunk, int64_t(V) + off)); };
    int passes = 0;
    uint64_t before = 0, mine = 0;  // sums of the parts before the CTA's, and its own, in the last pass

    // every CTA's value to all: the cluster's sum (and what lies before this CTA's part), or maximum
    auto meet = [&](uint64_t v, bool maximum) {
        if (tid == 0) sm.total[passes & 1] = v;
        cl.sync();
        // a lane per CTA: one after the other these loads take 0.3 us each
        const int c = tid % 32;
        const uint64_t w = c < C ? *cl.map_shared_rank(&sm.total[passes & 1], c) : 0;
        const uint64_t all = maximum ? warp_max(w) : p.capped ? warp_sum_capped(w) : warp_sum(w);
        if (!maximum) before = p.capped ? warp_sum_capped(c < rank ? w : 0) : warp_sum(c < rank ? w : 0);
        mine = v;
        ++passes;  // the other place next: who still reads this one is waited for there
        return all;
    };
    auto cta_total = [&](uint64_t v, bool maximum) {  // of the warps' values
        if (tid % 32 == 0) sm.warp[tid / 32] = v;
        __syncthreads();
        const uint64_t w = tid % 32 < kWarps ? sm.warp[tid % 32] : 0;
        return maximum ? warp_max(w) : p.capped ? warp_sum_capped(w) : warp_sum(w);
    };
    auto mass = [&](const Residual& r) {
        uint64_t sum = 0, all = 0;
        int hi = 0, lo = 0;  // of a step
        const int off = offset(r.p), last = end_of(off);
        auto step = [&]() {
            sum += uint64_t(int64_t(hi) * (1 << kHalf) + lo);
            hi = lo = 0;
        };
        auto add_p = [&](int, float x, float) {
            const Fixed P = halves(x);
            hi += P.hi, lo += P.lo;
        };
        auto add_diff = [&](int, float x, float y) {  // a = 1, which gives the same numbers
            const Fixed P = halves(x), Q = halves(y);
            if (__saturatef(x) > __saturatef(y)) hi += P.hi - Q.hi, lo += P.lo - Q.lo;
        };
        auto add = [&](int, float x, float y) {
            const Fixed S = less(x, y, r.a_hi, r.a_lo);
            hi += S.hi, lo += S.lo;
        };
        auto done = [&](int t) {
            sum = warp_sum(sum);
            if (r.n_gone) {  // refused tokens weigh nothing
                uint64_t away = 0;
                const int begin = first + t * p.tile;
                for (int k = tid % 32; k < r.n_gone; k += 32) {
                    bool again = false;
                    for (int j = 0; j < k; ++j) again |= r.gone[j] == r.gone[k];
                    if (!again && r.gone[k] + off >= begin && r.gone[k] + off < last && r.gone[k] + off - begin < p.tile)
                        away += uint64_t(r.of(__ldg(r.p + r.gone[k]), 0.0f));
                }
                sum -= warp_sum(away);
            }
            if (tid % 32 == 0) sm.tile[t] = sum;
            all += sum;
            if (p.capped) all = min(all, kTooMuch);
            sum = 0;
        };
        // the whole part on its way to L2 at once: the warps' own loads are a few rounds, each of which would wait for HBM
        if (tid < 2 && first < last && (tid == 0 || r.a_hi != 0.0f)) {
            const float* const row = tid == 0 ? r.p : r.q;
            const int o = offset(row), from = first > o ? first : 4, to = min(first + p.chunk, V + o) & ~3;
            if (from < to) prefetch_l2(row + (from - o), uint32_t(to - from) * 4);
        }
        __syncthreads();  // the tiles and the warps' words of the pass before are read
        if (r.a_hi == 0.0f)
            walk_row<false>(p, r.p, r.p, off, first, last, add_p, step, done);
        else if (r.a_hi == 1.0f && r.a_lo == 0.0f)
            walk_row<true>(p, r.p, r.q, off, first, last, add_diff, step, done);
        else
            walk_row<true>(p, r.p, r.q, off, first, last, add, step, done);
        return meet(cta_total(all, false), false);
    };
    __syncthreads();
    if (tid > 0 && tid < T && sm.par[tid] >= 0) atomicOr(&sm.kids[sm.par[tid]], 1ull << tid);
    if (tid == 0) sm.path[0] = 0;
    __syncthreads();

    int cur = 0, len = 1, next = -1;
    bool owner = rank == 0;  // who writes next
    for (;;) {
        const float* const prow = p.a.target + (t0 + int64_t(cur)) * p.a.target_ld;
        int taken = -1;
        unsigned long long kids = len < p.a.path_ld ? sm.kids[cur] : 0;  // in the order of their numbers
        if (greedy) {
            uint64_t best = 0;
            __syncthreads();
            walk_row<false>(
                p, prow, prow, offset(prow), first, end_of(offset(prow)),
                [&](int i, float x, float) {
                    const uint32_t o = ordered(x);
                    if (o > uint32_t(best >> 32) || (o && o == uint32_t(best >> 32) && uint32_t(~i) > uint32_t(best)))
                        best = uint64_t(o) << 32 | uint32_t(~i);
                },
                []() {}, [](int) {});
            best = meet(cta_total(warp_max(best), true), true);
            next = best ? int(~uint32_t(best)) : -1;
            for (; kids && taken < 0; kids &= kids - 1)
                if (sm.tok[__ffsll(kids) - 1] == next) taken = __ffsll(kids) - 1;
            if (taken < 0) break;
        } else {
            Residual r = {prow, p.a.draft ? p.a.draft + (t0 + int64_t(cur)) * p.a.draft_ld : nullptr, 0.0f, 0.0f, 0, sm.gone};
            double a = 0.0, W = 1.0;  // thread 0's: fp64 of a whole CTA takes 16 cycles per warp and instruction
            uint64_t mass_fixed = 0;
            bool known = false;  // mass_fixed and the tiles are of r as it stands
            for (;;) {
                __syncthreads();
                if (tid == 0) {
                    sm.act = kEnd;
                    for (; kids; kids &= kids - 1) {
                        const int c = __ffsll(kids) - 1, x = sm.tok[c];
                        double S = double(sm.p[c]) - a * double(sm.q[c]);
                        if (!r.q)
                            for (int k = 0; k < r.n_gone; ++k)
                                if (sm.gone[k] == x) S = 0.0;
                        if (S > 0.0 && double(sm.u[c]) * double(sm.q[c]) * W < S) {
                            sm.act = kAccept, sm.child = c;
                            break;
                        }
                        if (r.q) {
                            if (known && mass_fixed == 0) continue;  // nothing is left to accept, or to take away
                            a += W;
                            sm.a_hi = float(a);
                            sm.a_lo = float(a - double(sm.a_hi));
                            sm.act = kRefuse;
                            kids &= kids - 1;
                            break;
                        }
                        W -= S > 0.0 ? S : 0.0;
                        sm.gone[r.n_gone++] = x;
                    }
                    sm.n_gone = r.n_gone;
                }
                __syncthreads();
                const int act = sm.act;
                r.n_gone = sm.n_gone;
                if (act == kAccept) taken = sm.child;
                if (act != kRefuse) break;
                r.a_hi = sm.a_hi, r.a_lo = sm.a_lo;
                mass_fixed = mass(r);
                if (tid == 0) W = double(mass_fixed) * kInvOne;
                known = true;
                if (mass_fixed >= kTooMuch) break;
            }
            if (taken < 0) {
                if (!known) mass_fixed = mass(r);
                if (mass_fixed == 0 && (r.a_hi != 0.0f || r.n_gone)) {  // the target's row itself where the residual is empty
                    r.a_hi = 0.0f, r.n_gone = 0;
                    mass_fixed = mass(r);
                }
                if (mass_fixed >= kTooMuch && rank == 0 && tid == 0) atomicOr(status, MQ_DEV_KV_RANGE);
                if (mass_fixed == 0 || mass_fixed >= kTooMuch) break;
                // the first index whose running sum passes u W
                const uint64_t u = fixed(sm.u[0]), U = u < (1ull << kOne) ? u : (1ull << kOne) - 1;
                const uint64_t mark = __umul64hi(U << (64 - kOne), mass_fixed);
                owner = int64_t(mark) >= int64_t(before) && int64_t(mark - before) < int64_t(mine);
                if (owner) {
                    uint64_t at = before;
                    const int off = offset(r.p), last = end_of(off);
                    if (tid < 32) {
                        // the tile, 32 at a time, then 32 runs of 16 of each of its units
                        const int tiles = (last - first + p.tile - 1) / p.tile;
                        int t = -1;
                        for (int b = 0; b < tiles && t < 0; b += 32) {
                            uint64_t incl = b + tid < tiles ? sm.tile[b + tid] : 0;
                            const uint64_t own = incl;
#pragma unroll
                            for (int o = 1; o < 32; o <<= 1) {
                                const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                                if (tid >= o) incl += v;
                            }
                            const unsigned past = __ballot_sync(0xffffffffu, int64_t(at + incl) > int64_t(mark));
                            const int l = past ? __ffs(past) - 1 : 31;
                            at += __shfl_sync(0xffffffffu, past ? incl - own : incl, l);
                            if (past) t = b + l;
                        }
                        const int begin = first + t * p.tile, end = last - begin < p.tile ? last : begin + p.tile;
                        for (int i = begin; i < end; i += kUnit) {
                            uint64_t own = 0;
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (i + tid * 16 + j >= off && i + tid * 16 + j < end) own += uint64_t(r.at(i + tid * 16 + j - off));
                            uint64_t incl = own;
#pragma unroll
                            for (int o = 1; o < 32; o <<= 1) {
                                const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                                if (tid >= o) incl += v;
                            }
                            const unsigned past = __ballot_sync(0xffffffffu, int64_t(at + incl) > int64_t(mark));
                            if (!past) {
                                at += __shfl_sync(0xffffffffu, incl, 31);
                                continue;
                            }
                            if (tid == __ffs(past) - 1) {
                                uint64_t c = at + incl - own;
                                for (int j = 0; j < 16; ++j) {
                                    if (i + tid * 16 + j < off) continue;
                                    if (i + tid * 16 + j >= end) break;
                                    c += uint64_t(r.at(i + tid * 16 + j - off));
                                    if (int64_t(c) > int64_t(mark)) {
                                        sm.found = i + tid * 16 + j - off;
                                        break;
                                    }
                                }
                            }
                            break;
                        }
                    }
                    __syncthreads();
                    next = sm.found;
                }
                break;
            }
        }
        cur = taken;
        if (tid == 0) sm.path[len] = cur;
        ++len;
    }
    __syncthreads();
    if (rank == 0) {
        for (int i = tid; i < p.a.path_ld; i += kThreads) p.a.path[int64_t(s) * p.a.path_ld + i] = i < len ? sm.path[i] : 0;
        if (tid == 0) p.a.n_path[s] = len;
    }
    if (owner && tid == 0) p.a.next[s] = next;
    cl.sync();  // what the others still read of this CTA's shared memory
}

}  // namespace

cudaError_t set_verify_attributes()
{
    return cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t launch_verify(const mq_verify_args& a, int num_sms, unsigned* status, cudaStream_t s)
{
    VerifyArgs p;
    p.a = a;
    p.capped = a.vocab >= 1 << 18;
    // a step of every warp for each CTA at least; sixteen of them only for few sequences, since a larger cluster waits
    // for a whole neighbourhood of SMs
    int C = int64_t(a.n_seqs) * kMaxCluster <= num_sms ? kMaxCluster : kMaxCluster / 2;
    while (C > 1 && a.vocab <= (C / 2) * kUnit * kWarps) C /= 2;
    const int64_t part = (int64_t(a.vocab) + 3 + C - 1) / C;
    const int64_t units = (part + kUnit - 1) / kUnit;
    p.tile = int((units + kMaxTiles - 1) / kMaxTiles) * kUnit;
    p.chunk = int((part + p.tile - 1) / p.tile) * p.tile;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.n_seqs) * C);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel, p, status);
}

}  // namespace mq
