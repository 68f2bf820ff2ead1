// attn.cu -- attention of few query rows per key/value head (plain decoding
// and small trees) over the paged cache, on warp-level MMAs.
//
// Per (token, head): s_j = scale * q.k_j over the keys the node sees,
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), in one pass over the keys
// with a running maximum m.
//
// What bounds it is the cache's bytes, each of which is used once; the query
// rows of a key/value head (8 or 16 of them, tokens x group) ride along.  So:
// * one CTA per SM and an equal share of all pages for each (mq_attn.cuh);
//   whole (page, head) blocks come by one bulk copy each into a ring that
//   fills the shared memory.  One warp plans the segments ahead (divisions, the
//   page table's latency), one or two issue the copies;
// * the teams of four warps take the CTA's pages in turn.  In a page's 64 keys
//   each warp forms the scores of 16; the probabilities go round the team
//   through shared memory, and each warp sums a quarter of the head's values
//   over all 64, so a team holds one set of outputs, not four;
// * both products are formed transposed, keys and head values on the MMA's
//   16-row side and the query rows on its 8-column side, so 7 rows of a group
//   of 7 fill it: S^T[key][row] = K q^T, O^T[d][row] = V^T P^T.  The inner
//   index of an MMA may be permuted freely, so a lane takes its K values as
//   16-byte runs of two rows; S^T becomes P's operand by one 8x8 transpose per
//   8 keys.  q8_0 codes become f16 in registers on the way (byte permute,
//   exact subtraction, one rounded product with the scale);
// * the probabilities are rounded to f16 for the second product (2^-11 each,
//   the output's own rounding; a 32-bit operand would halve the MMAs' rate and
//   double what goes round the team), scaled by 2^10 so that a key at 2^-24 of
//   the largest still has a normal number, and their sum is formed from the
//   same rounded numbers by an MMA with ones, so the weights add up to one.
//   Root mean square error against 64 bits, relative: 2.6e-4 over 1000 keys,
//   2.9e-4 over 131071, where a result that is only rounded once has 2.1e-4;
// * the maximum is raised only when a score passes it by more than 5 (in
//   powers of two; 2^15 still fits f16), which after the first tiles is rare:
//   a predicate on the barrier that the team needs anyway, instead of a
//   maximum over its lanes and a rescaling;
// * a team that is done with a segment leaves its outputs in shared memory and
//   goes on to the next; a warp of its own joins them.  (Joined by the last team
//   to leave, the slowest fell behind further with every segment.)
// Scores, maxima, sums and outputs are fp32 throughout.
//
// Measured (28 query heads on 4 of 128, one token per sequence): 131071 tokens
// in f16 49.7 us, 5.4 TB/s, and 64 sequences of 128 to 8191 in f16 87 us,
// 6.2 TB/s: the cache's bytes.  The same 64 in q8_0 58 us, 5.0 TB/s: start
// and end of the call (about 10 us), and between them a page's instructions
// (about 300 of a warp's 500 convert; three teams are as fast as four), 0.53
// issued per cycle and scheduler: of a warp's waits per issue 1.6 are for
// loads, 1.5 for fixed latencies, 1.0 for instructions.  1000 tokens 9.9 us:
// latencies, of which the launch and the split take about 4, a page's copy 1,
// a page's products 1, and the two joins 4.
#include "mq_attn.cuh"

namespace mq {

namespace {

constexpr int kTeam = 4;  // warps that share a page
constexpr int kSegs = 4;  // segment descriptors in flight
constexpr int kMaxStages = 16;
constexpr int kRowsSmem = 218 * 1024;  // dynamic; the kernel's static arrays come on top
constexpr float kRaise = 5.0f, kShift = 10.0f, kLowest = -3.402823466e38f;

// what the producer hands over with a segment, besides its query rows
struct RowsSegment {
    AttnSegment g;
    int it0;  // number of its first page among the CTA's
};

// query rows 8*NT
template <int D, bool Q8, int NT>
struct RowsCfg {
    using B = KvBlock<D, Q8>;
    static constexpr int kRows = 8 * NT;
    static constexpr bool kJoins = NT == 1;  // the CTA that comes last joins a shared group
    // registers allow 16 warps of 8 rows or 12 of 16; the ring of 32 KB blocks is too short for four teams
    static constexpr int kTeams = D == 128 && (NT == 2 || !Q8) ? 3 : 4;
    static constexpr int kWarps = kTeams * kTeam;
    // Warps that copy pages, in turn: a page takes one 500 to 700 cycles whatever its size is, which is more than the
    // teams take for one of 9 or 17 KB, and less than one of 32 KB takes to come.
    static constexpr int kCopiers = B::kBytes < 32768 ? 2 : 1;
    static constexpr int kThreads = 32 * (kWarps + 2 + kCopiers);  // and the warps that plan, join and copy
    static constexpr int kSlice = D / kTeam;                     // head values that a warp sums
    static constexpr int kQ = kRows * D * 2;                     // a segment's query rows
    static constexpr int kP = NT * kTeam * 32 * 8;               // a page's probabilities
    static constexpr int kOut = kRows * D * 4;                   // a team's outputs
    static constexpr int kFixed = kSegs * kQ + kTeams * 2 * kP + 2 * kTeams * kOut;
    static constexpr int kFit = (kRowsSmem - kFixed) / B::kBytes;
    // A place belongs to one copier, so their number is even: teams of odd pages do not wait for those of even ones,
    // so the odd pages' copier can be a whole round of the ring ahead, where a wait by parity would not see that the
    // other's page has not even been there.
    static constexpr int kStages = (kFit < kMaxStages ? kFit : kMaxStages) / kCopiers * kCopiers;
    static constexpr int kSmem = kStages * B::kBytes + kFixed;
    static_assert(kStages > kTeams, "the teams' pages and one on its way");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16u(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

// more bytes to come in the barrier's phase, without an arrival
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ int load_acquire(const int* p)
{
    int v;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int* p, int v)
{
    asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}

// transpose of an 8x8 matrix of 16-bit values, lane l holding row l/4, columns 2(l%4), +1
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr uint32_t k64 = 0x64646464u;

// Lane (g = lane/4, t = lane%4).  K values of MMA step j: head values kdim(t, j) + 0..3.
template <int D, bool Q8>
__device__ __forceinline__ constexpr int kdim(int t, int j)
{
    return Q8 && D == 128 ? 32 * t + 4 * j : 64 * (j / 4) + 16 * t + 4 * (j % 4);
}

template <int D, int NT>
struct RowState {
    float o[NT][D / 64][4];  // values of output tile i: slice + (D/32) g + 2i, +1, of rows 2t, 2t + 1
    float l[NT][4];          // sums over the warp's own keys (every row of the ones-product is the same)
    float m[NT][2];          // running maxima of rows 2t, 2t + 1, the same in the whole team
};

// A tile that reaches past the context, before its values are used: rows past
// the sequence's end become zeros, and so do values that are not finite, since
// 0 * NaN would reach rows that do not see the key; those values are added to
// the outputs of the rows that do (whatever a key's weight is, they make the
// output what they are).  The warp owns the tile's rows of the stage.
template <int D, bool Q8>
__device__ __noinline__ bool clean_values(uint8_t* blk, int r0, int key0, int len)  // true: not finite ones remain
{
    using B = KvBlock<D, Q8>;
    const int lane = threadIdx.x & 31;
    bool suspect = false;
    if (Q8) {
        // codes are finite; a product with the scale overflows only above 65504 / 127
        __half* const sc = reinterpret_cast<__half*>(blk + B::kScK + B::kScBytes) + r0 * (D / 32);
        for (int i = lane; i < 16 * (D / 32); i += 32) {
            if (key0 + i / (D / 32) >= len)
                sc[i] = __ushort_as_half(0);
            else
                suspect |= !(fabsf(__half2float(sc[i])) < 512.0f);
        }
    } else {
        for (int i = lane; i < 16 * (D / 8); i += 32) {
            const int r = i / (D / 8);
            uint4* const x = reinterpret_cast<uint4*>(blk + B::kVOff + B::chunk(r0 + r, i % (D / 8)));
            if (key0 + r >= len) {
                *x = make_uint4(0, 0, 0, 0);
            } else {
                const uint4 v = *x;  // exponent bits all ones carry into the sign's place
                const uint32_t m = 0x7c007c00u, a = 0x04000400u;
                suspect |= ((((v.x & m) + a) | ((v.y & m) + a) | ((v.z & m) + a) | ((v.w & m) + a)) & 0x80008000u) != 0;
            }
        }
    }
    return __any_sync(0xffffffffu, suspect);
}

// zeroes the tile's values that are not finite
template <int D, bool Q8>
__device__ __noinline__ void drop_values(uint8_t* blk, int r0)
{
    using B = KvBlock<D, Q8>;
    const int lane = threadIdx.x & 31;
    for (int r = r0; r < r0 + 16; ++r) {
        uint32_t drop = 0;
        for (int e = 0; e < D / 32; ++e) {
            const float v = kv_value<D, Q8>(blk, r, lane + 32 * e, 1);
            drop |= !(v - v == 0.0f) ? 1u << e : 0u;
        }
        __syncwarp();
        for (int e = 0; e < D / 32; ++e) {
            const int d = lane + 32 * e;
            if (Q8) {  // the code of zero, and a finite scale
                if (drop >> e & 1) blk[B::kVOff + B::chunk(r, d >> 4) + (d & 15)] = 128;
                __half* const sc = reinterpret_cast<__half*>(blk + B::kScK + B::kScBytes) + r * (D / 32) + e;
                if (lane == 0 && !(fabsf(__half2float(*sc)) <= 65504.0f)) *sc = __ushort_as_half(0);
            } else if (drop >> e & 1) {
                *reinterpret_cast<uint16_t*>(blk + B::kVOff + B::chunk(r, d >> 3) + (d & 7) * 2) = 0;
            }
        }
    }
    __syncwarp();
}

// A lane's places in a block, in bytes from its start, for the scores of rows
// r0.. and the values of slice w of rows 0..15 (the rows 8 and 16 further have
// the same permutation, so their places are constants away).
template <int D, bool Q8>
struct PagePlaces {
    using B = KvBlock<D, Q8>;
    uint32_t k, sk;   // first 16-byte run of K row r0 + g (the next is at ^ 16), its scale (q8_0)
    uint32_t v0, v1;  // the lane's D/32 values of V rows 2t and 2t + 1
    uint32_t sv;      // q8_0: scales of V rows 2 * lane, + 1
    __device__ __forceinline__ PagePlaces(int r0, int w, int lane)
    {
        const int g = lane >> 2, t = lane & 3, ra = r0 + g;
        if (Q8) {
            k = B::chunk(ra, (D / 64) * t);
            sk = B::kScK + (ra * (D / 32) + (D == 128 ? t : t >> 1)) * 2;
            const int d = w * (D / 4) + g * (D / 32);
            v0 = B::kVOff + B::chunk(2 * t, d >> 4) + (d & 15);
            v1 = B::kVOff + B::chunk(2 * t + 1, d >> 4) + (d & 15);
            sv = B::kScK + B::kScBytes + (2 * lane * (D / 32) + (w * (D / 4) >> 5)) * 2;
        } else {
            k = B::chunk(ra, 2 * t);
            const int d = w * (D / 4) + g * (D / 32);
            v0 = B::kVOff + B::chunk(2 * t, d >> 3) + (d & 7) * 2;
            v1 = B::kVOff + B::chunk(2 * t + 1, d >> 3) + (d & 7) * 2;
            sk = sv = 0;
        }
    }
};

enum { kFlagRaise = 1, kFlagOdd = 2, kFlagFail = 4 };

// a team's words in shared memory
template <int NT>
struct TeamWords {
    float top[kTeam][8 * NT];  // the warps' maxima when the team's is raised
    int flags;
};

// ---- one page ------------------------------------------------------------------------------
// ok: the page is there (false goes round the team, which gives up together).
// p_at: the team's probabilities of this page (every other page has the other place).
template <int D, bool Q8, int NT>
__device__ __forceinline__ bool rows_page(bool ok, uint8_t* blk, int wi, int team, int page_key, const PagePlaces<D, Q8>& at,
                                          const uint32_t (&q)[NT][D / 16][2], float scale_log2, RowState<D, NT>& st,
                                          int ctx, int len, const uint64_t* row_mask, uint2* p_at, TeamWords<NT>* words)
{
    using B = KvBlock<D, Q8>;
    constexpr int k8 = 8 * B::kRow;          // eight rows on
    constexpr int s8 = 8 * (D / 32) * 2;     // their scales
    constexpr int kPlane = kKvPage * 128;    // f16: the next 64 values
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, id = 2 + team;
    const uint32_t base = smem_u32(blk);
    const int r0 = 16 * wi, key0 = page_key + r0;
    const bool tail = page_key + kKvPage > ctx;  // visibility is tested key by key
    // ---- S^T of the warp's 16 keys
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
    if constexpr (Q8) {
        const uint32_t da = lds16u(base + at.sk) * 0x10001u, db = lds16u(base + at.sk + s8) * 0x10001u;
        constexpr int LD = D / 64;  // 16-byte runs of a lane per row
#pragma unroll
        for (int h = 0; h < LD; ++h) {
            const uint32_t ka = (base + at.k) ^ (h << 4);  // blocks start at multiples of 128
            const uint4 xa = lds128(ka), xb = lds128(ka + k8);
            const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t a0 = kv_pair(__byte_perm(wa[w], k64, 0x4140), da);
                const uint32_t a1 = kv_pair(__byte_perm(wb[w], k64, 0x4140), db);
                const uint32_t a2 = kv_pair(__byte_perm(wa[w], k64, 0x4342), da);
                const uint32_t a3 = kv_pair(__byte_perm(wb[w], k64, 0x4342), db);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(s[n], a0, a1, a2, a3, q[n][4 * h + w][0], q[n][4 * h + w][1]);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {  // plane h/2, chunk 2t + h%2: 8 values, two MMA steps
            const uint32_t ka = ((base + at.k) ^ ((h & 1) << 4)) + (h >> 1) * kPlane;
            const uint4 xa = lds128(ka), xb = lds128(ka + k8);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16816(s[n], xa.x, xb.x, xa.y, xb.y, q[n][2 * h][0], q[n][2 * h][1]);
                mma16816(s[n], xa.z, xb.z, xa.w, xb.w, q[n][2 * h + 1][0], q[n][2 * h + 1][1]);
            }
        }
    }
    bool raise = false, odd = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] *= scale_log2;
        if (tail) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = key0 + g + (e >> 1) * 8;
                const uint64_t bits = row_mask[8 * n + 2 * t + (e & 1)];
                if (!(j < ctx || (j < len && ((bits >> (j - ctx)) & 1)))) s[n][e] = -INFINITY;
            }
        }
        raise |= fmaxf(s[n][0], s[n][2]) > st.m[n][0] + kRaise || fmaxf(s[n][1], s[n][3]) > st.m[n][1] + kRaise;
    }
    if (tail && ok && key0 < len) odd = clean_values<D, Q8>(blk, r0, key0, len);
    // ---- softmax numerators, round the team
    uint32_t pb[NT][2];
    auto numerators = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float m0 = st.m[n][0] - kShift, m1 = st.m[n][1] - kShift;
            pb[n][0] = transpose8x8(pack_f16(ex2(s[n][0] - m0), ex2(s[n][1] - m1)));
            pb[n][1] = transpose8x8(pack_f16(ex2(s[n][2] - m0), ex2(s[n][3] - m1)));
            p_at[(n * kTeam + wi) * 32 + lane] = make_uint2(pb[n][0], pb[n][1]);
        }
    };
    numerators();
    const int flags = (__any_sync(0xffffffffu, raise) ? kFlagRaise : 0) | (odd ? kFlagOdd : 0) | (ok ? 0 : kFlagFail);
    if (flags && lane == 0) atomicOr(&words->flags, flags);
    if (barrier_any(id, 32 * kTeam, flags != 0)) {
        // ---- rare, and the whole team together
        const int all = *const_cast<volatile int*>(&words->flags);
        named_barrier_sync(id, 32 * kTeam);
        if (wi == 0 && lane == 0) words->flags = 0;
        if (all & kFlagFail) return false;
        if (all & kFlagOdd) {
            // whatever a key's weight is, a value that is not finite makes the outputs of the
            // rows that see it what it is; then it is dropped, for the rows that do not
#pragma unroll 1
            for (int r = 0; r < min(kKvPage, len - page_key); ++r) {
                const int j = page_key + r;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint64_t bits = row_mask[8 * n + 2 * t + e];
                        if (!(j < ctx || ((bits >> (j - ctx)) & 1))) continue;
#pragma unroll
                        for (int i = 0; i < D / 64; ++i)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float v = kv_value<D, Q8>(blk, r, wi * (D / 4) + (D / 32) * g + 2 * i + x, 1);
                                if (!(v - v == 0.0f)) st.o[n][i][e + 2 * x] += v;
                            }
                    }
            }
            named_barrier_sync(id, 32 * kTeam);
            if (key0 < len) drop_values<D, Q8>(blk, r0);
        }
        if (all & kFlagRaise) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                    if (g == 0) words->top[wi][8 * n + 2 * t + e] = x;
                }
            named_barrier_sync(id, 32 * kTeam);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mn = st.m[n][e];
#pragma unroll
                    for (int w = 0; w < kTeam; ++w) mn = fmaxf(mn, words->top[w][8 * n + 2 * t + e]);
                    const float f = attn_factor(st.m[n][e] - mn);
                    st.m[n][e] = mn;
                    st.l[n][e] *= f;
                    st.l[n][e + 2] *= f;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        st.o[n][i][e] *= f;
                        st.o[n][i][e + 2] *= f;
                    }
                }
            numerators();
        }
        named_barrier_sync(id, 32 * kTeam);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        constexpr uint32_t one = 0x3c003c00u;
        mma16816(st.l[n], one, one, one, one, pb[n][0], pb[n][1]);
    }
    // ---- O^T of the warp's slice over the page's keys, 16 a step: keys 2t, 2t + 1, 2t + 8, 2t + 9
    uint32_t dv = 0;
    if (Q8) dv = __byte_perm(lds16u(base + at.sv), lds16u(base + at.sv + (D / 32) * 2), 0x5410);
#pragma unroll
    for (int ks = 0; ks < kTeam; ++ks) {
        if (tail && page_key + 16 * ks >= len) break;  // rows that were not cleaned
        uint2 p2[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) p2[n] = p_at[(n * kTeam + ks) * 32 + lane];
        auto product = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(st.o[n][i], a0, a1, a2, a3, p2[n].x, p2[n].y);
        };
        const uint32_t va = base + at.v0 + 2 * ks * k8, vb = base + at.v1 + 2 * ks * k8;
        if constexpr (Q8) {
            const uint32_t d01 = __shfl_sync(0xffffffffu, dv, 8 * ks + t), d23 = __shfl_sync(0xffffffffu, dv, 8 * ks + t + 4);
            if constexpr (D == 128) {
                const uint32_t x0 = lds32(va), x1 = lds32(vb), x2 = lds32(va + k8), x3 = lds32(vb + k8);
                const uint32_t pl = __byte_perm(x0, x1, 0x5140), ph = __byte_perm(x0, x1, 0x7362);
                const uint32_t rl = __byte_perm(x2, x3, 0x5140), rh = __byte_perm(x2, x3, 0x7362);
                product(0, kv_pair(__byte_perm(pl, k64, 0x4140), d01), kv_pair(__byte_perm(pl, k64, 0x4342), d01),
                        kv_pair(__byte_perm(rl, k64, 0x4140), d23), kv_pair(__byte_perm(rl, k64, 0x4342), d23));
                product(D / 64 - 1, kv_pair(__byte_perm(ph, k64, 0x4140), d01), kv_pair(__byte_perm(ph, k64, 0x4342), d01),
                        kv_pair(__byte_perm(rh, k64, 0x4140), d23), kv_pair(__byte_perm(rh, k64, 0x4342), d23));
            } else {
                const uint32_t pl = __byte_perm(lds16u(va), lds16u(vb), 0x5140);
                const uint32_t rl = __byte_perm(lds16u(va + k8), lds16u(vb + k8), 0x5140);
                product(0, kv_pair(__byte_perm(pl, k64, 0x4140), d01), kv_pair(__byte_perm(pl, k64, 0x4342), d01),
                        kv_pair(__byte_perm(rl, k64, 0x4140), d23), kv_pair(__byte_perm(rl, k64, 0x4342), d23));
            }
        } else if constexpr (D == 128) {
            const uint2 x0 = lds64(va), x1 = lds64(vb), x2 = lds64(va + k8), x3 = lds64(vb + k8);
            product(0, __byte_perm(x0.x, x1.x, 0x5410), __byte_perm(x0.x, x1.x, 0x7632), __byte_perm(x2.x, x3.x, 0x5410),
                    __byte_perm(x2.x, x3.x, 0x7632));
            product(D / 64 - 1, __byte_perm(x0.y, x1.y, 0x5410), __byte_perm(x0.y, x1.y, 0x7632),
                    __byte_perm(x2.y, x3.y, 0x5410), __byte_perm(x2.y, x3.y, 0x7632));
        } else {
            const uint32_t x0 = lds32(va), x1 = lds32(vb), x2 = lds32(va + k8), x3 = lds32(vb + k8);
            product(0, __byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x7632), __byte_perm(x2, x3, 0x5410),
                    __byte_perm(x2, x3, 0x7632));
        }
    }
    // the next bulk copy into this stage comes after the cleaning's writes
    if (tail) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return true;
}

// ---- the kernel ----------------------------------------------------------------------------
template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(RowsCfg<D, Q8, NT>::kThreads, 1)
    attn_rows_kernel(const AttnParams p, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    using C = RowsCfg<D, Q8, NT>;
    constexpr int RT = C::kRows, kCopiers = C::kCopiers, kTeams = C::kTeams, kWarps = C::kWarps, kStages = C::kStages;
    extern __shared__ __align__(128) uint8_t sm[];
    uint8_t* const ring = sm;
    __half* const q_s = reinterpret_cast<__half*>(sm + kStages * B::kBytes);
    uint2* const p_s = reinterpret_cast<uint2*>(sm + kStages * B::kBytes + kSegs * C::kQ);
    float* const out_s = reinterpret_cast<float*>(sm + kStages * B::kBytes + kSegs * C::kQ + kTeams * 2 * C::kP);
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], seg_planned[kSegs], seg_full[kSegs], seg_empty[kSegs];
    __shared__ __align__(8) uint64_t out_full[2], out_free[2], part_done[2];
    __shared__ AttnSegment split_s[2];  // the groups that it shares
    __shared__ int last_s[2];
    __shared__ RowsSegment seg_s[kSegs];
    __shared__ uint64_t mask_s[kSegs][RT];
    __shared__ int32_t pages_s[kSegs][32];  // a segment's first ones
    // a segment's teams (every other segment has the other place): maxima, sums, whether there were pages, bad ones
    __shared__ float m_s[2][kTeams][RT], l_s[2][kTeams][kTeam][RT];
    __shared__ int had_s[2][kTeams];
    __shared__ TeamWords<NT> words_s[kTeams];
    __shared__ int bad_s[kStages], seen_s[kStages];
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x < kStages) {
        mbar_init(&full[threadIdx.x], 1);
        mbar_init(&empty[threadIdx.x], kTeam);
        seen_s[threadIdx.x] = 0;
    } else if (threadIdx.x >= 32 && threadIdx.x < 32 + kSegs) {
        mbar_init(&seg_planned[threadIdx.x - 32], 1);
        mbar_init(&seg_full[threadIdx.x - 32], 1);
        mbar_init(&seg_empty[threadIdx.x - 32], kWarps + 1 + kCopiers);
    } else if (threadIdx.x >= 64 && threadIdx.x < 66) {
        const int k = threadIdx.x - 64;
        mbar_init(&out_full[k], kWarps);
        mbar_init(&out_free[k], 1);
        mbar_init(&part_done[k], 1);
    } else if (threadIdx.x >= 96 && threadIdx.x < 96 + kTeams) {
        words_s[threadIdx.x - 96].flags = 0;
        if (threadIdx.x == 96) abort_flag = 0;
    }
    fence_barrier_init();
    if (!C::kJoins) griddep_launch_dependents();  // the join may take its place; it waits for this grid's end
    AttnRange w;
    if (warp == kWarps) w = attn_range(p, RT, status);
    __syncthreads();

    auto give_up = [&]() {
        abort_flag = 1;
        if (lane == 0) atomicOr(status, MQ_DEV_TIMEOUT);
    };
    // one outcome for the whole warp; after one wait that ran out, what is not there yet is not waited for
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait_bounded(bar, parity, p.limit_ns));
        if (!ok) give_up();
        return ok;
    };

    if (warp == kWarps) {
        // ---- the segments, ahead of the copies (a segment's set-up takes some microseconds: divisions, the page
        // table's latency, code that left the instruction cache)
        AttnSegment g = {};
        int at = w.first, it = 0, sg = 0;
        bool ok = true, more = true;
        int4 start[2] = {};  // the last segment's group, if it starts here and others go on with it
        for (; ok && more; ++sg) {
            more = attn_next(p, RT, &w, &at, &g);
            if (!more) g.n = g.T = 0;
            const int ss = sg % kSegs, rows = more ? min(RT, g.T * p.group - g.row0) : 0;
            const int32_t page = lane < g.n ? __ldg(p.c.table + int64_t(g.seq) * p.c.table_ld + g.page0 + lane) : 0;
            uint64_t bits = 0;
            const int row = g.row0 + lane, node = attn_row_token(p, row);
            if (lane < rows) bits = p.a.mask ? __ldg(p.a.mask + g.t0 + node) : ~0ull >> (63 - node);
            if (sg >= kSegs) ok = wait_all(&seg_empty[ss], uint32_t(sg / kSegs - 1) & 1u);
            if (!ok) break;
            if (more && g.n_ctas > 1 && g.cta0 == int(blockIdx.x)) attn_shared(g, start);
            if (lane == 0) {
                seg_s[ss].g = g;
                seg_s[ss].it0 = it;
            }
            pages_s[ss][lane] = page;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&seg_planned[ss]);
                mbar_expect_tx(&seg_full[ss], uint32_t(rows) * D * 2);
            }
            __syncwarp();
            if (lane < rows)
                bulk_copy_g2s(q_s + (ss * RT + lane) * D,
                              static_cast<const __half*>(p.a.q) + int64_t(g.t0 + node) * p.a.q_ld +
                                  ((g.head - node) * p.group + row) * D,
                              D * 2, &seg_full[ss]);
            if (lane < RT) mask_s[ss][lane] = bits;
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_full[ss]);
            it += g.n;
        }
        // every CTA says so in every call, one that gave up too: the join finds nothing of another call
        if (!C::kJoins && lane < 2) p.shared[2 * blockIdx.x + lane] = lane == 0 ? start[0] : start[1];
        // copies still in flight land before the CTA can exit
        for (int j = sg > kSegs ? sg - kSegs : 0; j < sg; ++j)
            (void)mbar_wait_bounded(&seg_full[j % kSegs], uint32_t(j / kSegs) & 1u, p.limit_ns);
        return;
    }

    if (warp >= kWarps + 2) {
        // ---- the pages' copies, by lane 0; the warp reads their numbers 32 at a time
        int it = warp - (kWarps + 2), s = it, total = -1;
        uint32_t phase = 0;
        bool ok = true;
        for (int sg = 0; ok; ++sg) {
            const int ss = sg % kSegs;
            ok = wait_all(&seg_planned[ss], uint32_t(sg / kSegs) & 1u);
            if (!ok) break;
            const AttnSegment& g = seg_s[ss].g;
            const int n = g.n, it0 = seg_s[ss].it0;
            if (n == 0) {
                total = it0;
                break;
            }
            const int withheld = p.withhold && sg == 0 ? it0 + n - 1 : -1;  // test-only fault
            const int32_t* const table = p.c.table + int64_t(g.seq) * p.c.table_ld + g.page0 + lane;
            const uint8_t* const src = p.c.pages + int64_t(g.head) * B::kBytes;
            int at = 0;  // the pages at .. at + 31 are in the lanes
            int32_t page_l = pages_s[ss][lane], next_l = 32 + lane < n ? __ldg(table + 32) : 0;
            for (; it < it0 + n; it += kCopiers) {
                if (it - it0 >= at + 32) {
                    at += 32;
                    page_l = next_l;
                    if (at + 32 + lane < n) next_l = __ldg(table + at + 32);
                }
                const int32_t page = __shfl_sync(0xffffffffu, page_l, it - it0 - at);
                if (it >= kStages) ok = wait_all(&empty[s], phase ^ 1u);
                if (!ok) break;
                if (lane == 0 && it != withheld) {
                    const bool bad = page < 0 || page >= p.c.n_pages;  // table entries are not trusted
                    bad_s[s] = bad;
                    if (bad) {
                        mbar_arrive(&full[s]);
                    } else {
                        mbar_arrive_expect_tx(&full[s], B::kBytes);
                        bulk_copy_g2s(ring + s * B::kBytes, src + int64_t(page) * p.c.n_kv_heads * B::kBytes, B::kBytes,
                                      &full[s]);
                    }
                }
                s += kCopiers;
                if (s >= kStages) s -= kStages, phase ^= 1u;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[ss]);
        }
        // its copies still in flight land before the CTA can exit (older ones' places have been used again)
        for (int j = it - kCopiers; j >= 0 && j >= (total < 0 ? it + 1 : total) - kStages; j -= kCopiers)
            (void)mbar_wait_bounded(&full[j % kStages], uint32_t(j / kStages) & 1u, p.limit_ns);
        return;
    }

    if (warp == kWarps + 1) {
        // ---- the segments' joins, in order, while the teams are at later ones
        int splits = 0;
        bool ok = true;
        for (int sg = 0;; ++sg) {
            const int ss = sg % kSegs, os = sg & 1;
            ok = wait_all(&seg_full[ss], uint32_t(sg / kSegs) & 1u);
            if (!ok || seg_s[ss].g.n == 0) break;  // (behind the last segment: no pages)
            ok = wait_all(&out_full[os], uint32_t(sg / 2) & 1u);
            if (!ok) break;
            const AttnSegment& g = seg_s[ss].g;
            const bool split = g.n_ctas > 1;
            const int rows = min(RT, g.T * p.group - g.row0);
            float* const slot = p.parts + (int64_t(blockIdx.x) * 2 + g.slot) * attn_slot_floats(RT, D);
            int had = 0;  // the teams that had pages
            bool bad = false;
#pragma unroll
            for (int k = 0; k < kTeams; ++k) {
                had |= had_s[os][k] != 0 ? 1 << k : 0;
                bad |= had_s[os][k] == 2;
            }
            // lane l: row l % 8 (+ 8j) of team l / 8: its weight, and the row's maximum and sum
            float fk[NT], top[NT], sum[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int k = lane >> 3, r = 8 * j + (lane & 7);
                const bool there = had >> k & 1;
                const float mk = there ? m_s[os][k][r] : kLowest;
                float lk = 0.0f;
#pragma unroll
                for (int u = 0; u < kTeam; ++u) lk += there ? l_s[os][k][u][r] : 0.0f;
                top[j] = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, 8));
                top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
                fk[j] = there ? attn_factor(mk - top[j]) : 0.0f;
                sum[j] = lk * fk[j];
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
                if (split && lane < 8 && r < rows) {
                    slot[r] = top[j];
                    slot[RT + r] = bad ? kAttnBadPage : sum[j];
                }
                sum[j] = sum[j] == 0.0f ? 0.0f : 1.0f / sum[j];
            }
            constexpr int kLanes = D / 4, kStep = 32 / kLanes;  // lanes of a row with four values each, rows at a time
            const int d = lane % kLanes * 4;
#pragma unroll
            for (int j = 0; j < RT; j += kStep) {
                if (j >= rows) break;
                const int r = j + lane / kLanes;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kTeams; ++k) {
                    const float f = __shfl_sync(0xffffffffu, fk[j / 8], 8 * k + (r & 7));
                    if (!(had >> k & 1)) continue;  // what lies there is not read as a number
                    const float4 o = *reinterpret_cast<const float4*>(out_s + ((os * kTeams + k) * RT + r) * D + d);
                    v.x = fmaf(o.x, f, v.x), v.y = fmaf(o.y, f, v.y), v.z = fmaf(o.z, f, v.z), v.w = fmaf(o.w, f, v.w);
                }
                const float inv = __shfl_sync(0xffffffffu, sum[j / 8], r & 7);
                if (split) {
                    if (r < rows) *reinterpret_cast<float4*>(slot + 2 * RT + r * D + d) = v;
                } else if (!bad) {
                    v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
                    attn_emit4(p, g, g.row0 + r, r < rows, D, d, v);
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&out_free[os]);
                if (!split && bad) atomicOr(status, MQ_DEV_KV_RANGE);
                if (C::kJoins && split) {
                    split_s[splits] = g;
                    last_s[splits] = attn_arrive(p, g);
                    mbar_arrive(&part_done[splits]);
                }
                mbar_arrive(&seg_empty[ss]);
            }
            splits += split;
        }
        if (!C::kJoins && !ok && lane < RT) {  // where the last CTA joins, a group without this one's arrival is not
            float* const slots = p.parts + int64_t(blockIdx.x) * 2 * attn_slot_floats(RT, D);
            slots[RT + lane] = slots[attn_slot_floats(RT, D) + RT + lane] = kAttnGaveUp;
        }
        if (C::kJoins && lane == 0) {  // the teams wait for two
            for (; splits < 2; ++splits) {
                last_s[splits] = 0;
                mbar_arrive(&part_done[splits]);
            }
        }
        return;
    }

    // ---- consumers
    const int team = warp / kTeam, wi = warp % kTeam, g8 = lane >> 2, t4 = lane & 3, id = 2 + team;
    TeamWords<NT>* const words = &words_s[team];
    const PagePlaces<D, Q8> places(16 * wi, wi, lane);
    auto wait_seen = [&](int* word, int value) {
        bool ok = __all_sync(0xffffffffu, load_acquire(word) >= value);
        if (!ok) {
            const uint64_t t0 = global_timer_ns();
            do {
                ok = __all_sync(0xffffffffu, load_acquire(word) >= value);
            } while (__any_sync(0xffffffffu, !ok && !abort_flag && global_timer_ns() - t0 < p.limit_ns));
        }
        if (!ok) give_up();
        return ok;
    };
    bool good = true;  // the whole team's
    int it = team, s = team, flip = 0;
    uint32_t phase = 0;
    for (int sg = 0;; ++sg) {
        const int ss = sg % kSegs, os = sg & 1;
        bool ok = wait_all(&seg_full[ss], uint32_t(sg / kSegs) & 1u);
        // the outputs' place is free once the segment before the last has been joined
        if (sg >= 2) ok = wait_all(&out_free[os], uint32_t(sg / 2 - 1) & 1u) && ok;
        good = !barrier_any(id, 32 * kTeam, !ok);
        if (!good) break;
        const AttnSegment& g = seg_s[ss].g;  // stays until this warp's arrival at seg_empty
        const int ctx = g.ctx, len = ctx + g.T, end = seg_s[ss].it0 + g.n, first_key = (g.page0 - seg_s[ss].it0) * kKvPage;
        if (g.n == 0) break;
        const bool had = it < end;
        bool bad = false;
        if (had) {
            RowState<D, NT> st;
            uint32_t q[NT][D / 16][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // rows past the block's hold what was there: they stay in their own columns
                const __half* const src = q_s + (ss * RT + 8 * n + g8) * D;
#pragma unroll
                for (int j = 0; j < D / 16; j += 2) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + kdim<D, Q8>(t4, j));
                    q[n][j][0] = v.x, q[n][j][1] = v.y, q[n][j + 1][0] = v.z, q[n][j + 1][1] = v.w;
                }
                st.m[n][0] = st.m[n][1] = kLowest;  // finite: a row without keys keeps zero sums
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    st.l[n][e] = 0.0f;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) st.o[n][i][e] = 0.0f;
                }
            }
#pragma unroll 1
            for (; it < end; it += kTeams) {
                // The stage's previous use may be another team's page, which may not even have
                // landed; a wait by parity tells two successive uses apart only, so that team's
                // word that it has comes first.
                if (kStages % kTeams) ok = it < kStages || wait_seen(&seen_s[s], it - kStages + 1);
                ok = ok && wait_all(&full[s], phase);
                if (kStages % kTeams && ok && wi == 0 && lane == 0) store_release(&seen_s[s], it + 1);
                bad |= ok && bad_s[s] != 0;
                good = rows_page<D, Q8, NT>(ok, ring + s * B::kBytes, wi, team, first_key + it * kKvPage, places, q,
                                            p.scale_log2, st, ctx, len, mask_s[ss],
                                            p_s + (team * 2 + flip) * (C::kP / 8), words);
                if (!good) break;
                flip ^= 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                s += kTeams;
                if (s >= kStages) s -= kStages, phase ^= 1u;
            }
            if (!good) break;
            // ---- leave the team's results
            float* const mine = out_s + (os * kTeams + team) * RT * D + wi * C::kSlice + g8 * (D / 32);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * n + 2 * t4 + e;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
                        *reinterpret_cast<float2*>(mine + r * D + 2 * i) = make_float2(st.o[n][i][e], st.o[n][i][e + 2]);
                    if (g8 == 0) {
                        if (wi == 0) m_s[os][team][r] = st.m[n][e];
                        l_s[os][team][wi][r] = st.l[n][e];
                    }
                }
        }
        if (wi == 0 && lane == 0) had_s[os][team] = had ? (bad ? 2 : 1) : 0;
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&out_full[os]);
            mbar_arrive(&seg_empty[ss]);
        }
    }

    // ---- the shared groups whose last CTA this is: their segments joined in CTA order
    if (!C::kJoins) return;
    constexpr int kCons = 32 * kWarps;
    for (int k = 0; good && k < 2; ++k) good = wait_all(&part_done[k], 0);
    if (barrier_any(1, kCons, !good)) return;  // a wait that ran out anywhere ends all
    for (int k = 0; k < 2; ++k) {
        if (!last_s[k]) continue;
        const AttnSegment& g = split_s[k];
        const int rows = min(RT, g.T * p.group - g.row0);
        // every copy has landed and been read: the ring is free
        float* const sums = reinterpret_cast<float*>(ring);  // [kWarps][RT][D], then maxima and sums [kWarps][RT]
        float* const cm = sums + kWarps * RT * D;
        float* const cl = cm + kWarps * RT;
        // warp w joins the parts of CTAs w, w + kWarps, ...: lane r has row r's maximum and sum, and a
        // lane four values of each 128 of the rows
        constexpr int NV = RT * D / 128;
        float mr = kLowest, lr = 0.0f;
        bool gone = false;
        float4 acc[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int c = warp; c < g.n_ctas; c += kWarps) {
            const float* const slot =
                p.parts + (int64_t(g.cta0 + c) * 2 + (c == 0 ? g.slot0 : 0)) * attn_slot_floats(RT, D);
            const float mc = lane < rows ? __ldcg(slot + lane) : kLowest;
            const float lc = lane < rows ? __ldcg(slot + RT + lane) : 0.0f;
            float4 x[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v)
                x[v] = (v * 128 + lane * 4) / D < rows
                           ? __ldcg(reinterpret_cast<const float4*>(slot + 2 * RT) + lane + v * 32)
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            gone |= lc < 0.0f;
            const float mn = fmaxf(mr, mc), fr = attn_factor(mr - mn), fc = attn_factor(mc - mn);
            mr = mn;
            lr = lr * fr + lc * fc;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int r = (v * 128 + lane * 4) / D;
                const float a = __shfl_sync(0xffffffffu, fr, r), b = __shfl_sync(0xffffffffu, fc, r);
                acc[v].x = fmaf(acc[v].x, a, x[v].x * b);
                acc[v].y = fmaf(acc[v].y, a, x[v].y * b);
                acc[v].z = fmaf(acc[v].z, a, x[v].z * b);
                acc[v].w = fmaf(acc[v].w, a, x[v].w * b);
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            *reinterpret_cast<float4*>(sums + warp * RT * D + v * 128 + lane * 4) = acc[v];
        if (lane < RT) cm[warp * RT + lane] = mr, cl[warp * RT + lane] = lr;
        if (barrier_any(1, kCons, gone)) {  // a page outside the cache: the group stays unwritten
            if (threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
            continue;
        }
        // a warp per 128 values, four of a lane
        const int nw = min(kWarps, g.n_ctas);
        for (int x = warp * 128 + lane * 4; x - lane * 4 < rows * D; x += kWarps * 128) {
            const int r = x / D;
            float top = kLowest, sum = 0.0f;
#pragma unroll 8
            for (int u = 0; u < nw; ++u) top = fmaxf(top, cm[u * RT + r]);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
            for (int u = 0; u < nw; ++u) {
                const float f = attn_factor(cm[u * RT + r] - top);
                const float4 y = *reinterpret_cast<const float4*>(sums + u * RT * D + x);
                sum = fmaf(cl[u * RT + r], f, sum);
                v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
            attn_emit4(p, g, g.row0 + r, r < rows, D, x % D, v);
        }
        named_barrier_sync(1, kCons);
    }
}

// ---- the groups that several CTAs share: their parts joined in CTA order -------------------------
// A CTA per first CTA of a group.  A thread has four values of a row, of every kSplit-th of kJoinAhead parts; a
// group has some parts of 4 KB (16 at 1000 tokens, 38 at 16000 and more, with four key/value heads), which lie in
// L2, so what it costs is latency: all of a round's loads are on their way together, and before the maxima.
constexpr int kJoinAhead = 4;

template <int D, int NT>
struct RowsJoin {
    static constexpr int kRows = 8 * NT, kPart = kRows * D / 4;  // threads of a part
    static constexpr int kSplit = 1024 / kPart, kThreads = kPart * kSplit;
};

template <int D, int NT>
__global__ void __launch_bounds__(RowsJoin<D, NT>::kThreads) attn_rows_join_kernel(const AttnParams p, unsigned* status)
{
    using J = RowsJoin<D, NT>;
    constexpr int RT = J::kRows;
    constexpr int64_t kSlot = attn_slot_floats(RT, D);
    extern __shared__ float part_s[];  // [parts][RT] maxima, then sums
    __shared__ float4 sum_s[J::kSplit][J::kPart];
    const int cta0 = blockIdx.x, x = threadIdx.x % J::kPart, part = threadIdx.x / J::kPart;
    const int row = x / (D / 4), d = x % (D / 4) * 4;
    griddep_wait();
    const int4 s0 = __ldcg(p.shared + 2 * cta0), s1 = __ldcg(p.shared + 2 * cta0 + 1);
    const int n = s1.x;
    if (n < 2) return;
    AttnSegment g;
    g.t0 = s0.x, g.T = s0.y, g.head = s0.z, g.row0 = s0.w;
    const bool there = row < min(RT, g.T * p.group - g.row0);
    auto slot_of = [&](int c) { return p.parts + (int64_t(cta0 + c) * 2 + (c == 0 ? s1.y : 0)) * kSlot; };
    float4 v[kJoinAhead];
    auto load = [&](int c0) {
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
            v[i] = c0 + i < n && there ? __ldcg(reinterpret_cast<const float4*>(slot_of(c0 + i) + 2 * RT) + x)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    load(part * kJoinAhead);
    for (int i = threadIdx.x; i < 2 * RT * n; i += J::kThreads) {
        const int c = i / (2 * RT), k = i % (2 * RT);  // rows past the block's hold what was there, and stay theirs
        part_s[k < RT ? c * RT + k : n * RT + c * RT + k - RT] = __ldcg(slot_of(c) + k);
    }
    __syncthreads();
    float mm = kLowest, l = 0.0f;
    bool gone = false, bad = false;
    for (int c = 0; c < n; ++c) mm = fmaxf(mm, part_s[c * RT + row]);
    for (int c = 0; c < n; ++c) {
        const float lc = part_s[(n + c) * RT + row];
        gone |= there && lc < 0.0f;
        bad |= there && lc == kAttnBadPage;
        l = fmaf(lc, attn_factor(part_s[c * RT + row] - mm), l);
    }
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c0 = part * kJoinAhead; c0 < n;) {
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            if (c0 + i >= n) break;
            const float f = attn_factor(part_s[(c0 + i) * RT + row] - mm);
            o.x = fmaf(v[i].x, f, o.x), o.y = fmaf(v[i].y, f, o.y), o.z = fmaf(v[i].z, f, o.z), o.w = fmaf(v[i].w, f, o.w);
        }
        c0 += J::kSplit * kJoinAhead;
        if (c0 < n) load(c0);
    }
    sum_s[part][x] = o;
    if (__syncthreads_or(gone)) {  // the group stays unwritten
        if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    if (part > 0) return;
    for (int i = 1; i < min(J::kSplit, (n + kJoinAhead - 1) / kJoinAhead); ++i) {
        const float4 y = sum_s[i][x];
        o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    attn_emit4(p, g, g.row0 + row, there, D, d, o);
}

template <int D, bool Q8, int NT>
cudaError_t launch_rows(const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    using C = RowsCfg<D, Q8, NT>;
    attn_rows_kernel<D, Q8, NT><<<grid, C::kThreads, C::kSmem, s>>>(p, status);
    cudaError_t e = cudaGetLastError();
    if constexpr (!C::kJoins) {
        if (e == cudaSuccess && grid > 1)  // one CTA shares no group
            e = attn_launch_join(attn_rows_join_kernel<D, NT>, dim3(grid), RowsJoin<D, NT>::kThreads,
                                 size_t(grid) * 2 * C::kRows * sizeof(float), p, status, s);
    }
    return e;
}

template <int NT>
cudaError_t launch_rows_nt(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    if (c.type == MQ_TYPE_Q8_0)
        return c.head_dim == 128 ? launch_rows<128, true, NT>(p, grid, status, s)
                                 : launch_rows<64, true, NT>(p, grid, status, s);
    return c.head_dim == 128 ? launch_rows<128, false, NT>(p, grid, status, s)
                             : launch_rows<64, false, NT>(p, grid, status, s);
}

}  // namespace

// Workspace: what the join kernels read of the CTAs, the counters, parts.  Where each begins goes by the device alone,
// so a call finds the counters at zero whatever cache, sequences and rows the call before had.
static size_t parts_offset(int num_sms)
{
    return (size_t(num_sms) * (kAttnSharedBytes + sizeof(unsigned)) + 127) / 128 * 128;
}

// The most query rows of a key/value head that the warp kernels take.  16 rows, 8 key/value heads of 128, here and by
// attn_tc.cu: one sequence of 300 tokens, f16 11.6 and 11.7 us, q8_0 11.9 and 11.9; of 16000 25.3 and 25.8, 23.2 and
// 26.5; 16 of 100 to 3000 29 and 30, 27 and 34; 4 of 30000 84 and 86, 64 and 94.  Seven rows, 4 heads, one sequence of
// 300: 9.3 and 11.5, 9.2 and 11.8; 4 of 30000: 44 and 51, 30 and 55.
constexpr int kWarpRows = 16;

size_t attn_workspace_bytes(const mq_kv_cache& c, int n_heads, int max_tokens, int num_sms)
{
    const int RT = n_heads / c.n_kv_heads * max_tokens > kWarpRows ? attn_tc_rows() : kWarpRows;
    return parts_offset(num_sms) + size_t(num_sms) * 2 * attn_slot_floats(RT, c.head_dim) * sizeof(float);
}

cudaError_t launch_attn(const mq_kv_cache& cache, const mq_attn_args& a, void* ws, int num_sms, unsigned* status,
                        cudaStream_t s)
{
    AttnParams p;
    p.a = a;
    p.c = kv_view(cache);
    p.group = a.n_heads / cache.n_kv_heads;
    p.group_inv = uint32_t((0x100000000ull + p.group - 1) / p.group);
    p.scale_log2 = float(double(a.scale) * 1.4426950408889634);
    p.shared = static_cast<int4*>(ws);
    p.counters = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + size_t(num_sms) * kAttnSharedBytes);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + parts_offset(num_sms));
    p.limit_ns = uint64_t(fault_policy() == FAULT_NONE ? 2000 : 50) * 1000000ull;
    p.withhold = fault_policy() == FAULT_WITHHOLD_TILE;
    const int rows = p.group * a.max_tokens, RT = rows <= 8 ? 8 : rows <= kWarpRows ? 16 : attn_tc_rows();
    // no more CTAs than the bounds allow units
    const int64_t most = int64_t(cache.n_seqs) * ((int64_t(a.max_len) + kKvPage - 1) / kKvPage) * cache.n_kv_heads *
                         ((rows + RT - 1) / RT);
    const int grid = int(most < 1 ? 1 : most < num_sms ? most : num_sms);
    if (RT > kWarpRows) return launch_attn_tc(cache, p, grid, status, s);
    return RT == 8 ? launch_rows_nt<1>(cache, p, grid, status, s) : launch_rows_nt<2>(cache, p, grid, status, s);
}

cudaError_t set_attn_attributes(int max_smem)
{
    (void)max_smem;
    cudaError_t e = cudaSuccess;
#define MQ_SET(D, Q, N)                                                                                             \
    if (e == cudaSuccess)                                                                                           \
        e = cudaFuncSetAttribute(attn_rows_kernel<D, Q, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
    MQ_SET(128, true, 1) MQ_SET(64, true, 1) MQ_SET(128, false, 1) MQ_SET(64, false, 1)
    MQ_SET(128, true, 2) MQ_SET(64, true, 2) MQ_SET(128, false, 2) MQ_SET(64, false, 2)
#undef MQ_SET
    if (e == cudaSuccess) e = set_attn_tc_attributes();
    return e;
}

}  // namespace mq
