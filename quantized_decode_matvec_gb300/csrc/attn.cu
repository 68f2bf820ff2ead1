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
//   a producer lane brings whole (page, head) blocks by one bulk copy each
//   into a ring that fills the shared memory, and runs ahead over segments;
// * a page's 64 keys are four tiles of 16, one per warp of a team; the teams
//   take a segment's pages in turn;
// * both products are formed transposed, keys and head values on the MMA's
//   16-row side and the query rows on its 8-column side, so 7 rows of a group
//   of 7 fill it: S^T[key][row] = K q^T, O^T[d][row] = V^T P^T.  The inner
//   index of an MMA may be permuted freely, so a lane takes its K values as
//   16-byte runs of two rows, and its V values as 16-byte runs of the four
//   keys that its share of P needs; S^T becomes P's operand by one 8x8
//   transpose per 8 keys.  q8_0 codes become f16 in registers on the way
//   (byte permute, exact subtraction, one rounded product with the scale);
// * the probabilities are rounded to f16 for the second product (2^-11 each,
//   the output's own rounding), scaled by 2^10 so that a key at 2^-24 of the
//   largest still has a normal number, and their sum is formed from the same
//   rounded numbers by an MMA with ones, so the weights add up to one;
// * the maximum is raised only when a score passes it by more than 5 (in
//   powers of two; 2^15 still fits f16), which after the first tiles is rare:
//   a vote per tile instead of a maximum over its lanes and a rescaling.
// Scores, maxima, sums and outputs are fp32 throughout.
#include "mq_attn.cuh"

namespace mq {

namespace {

constexpr int kTeam = 4;       // warps that share a page
constexpr int kSegs = 4;       // segment descriptors in flight
constexpr int kMaxStages = 16;
constexpr float kRaise = 5.0f, kShift = 10.0f;

// query rows 8*NT.  Registers set the warps: with the producer 13 (NT = 1) may have 128 each, 9 (NT = 2) 168
template <int NT>
struct RowsCfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kTeams = NT == 1 ? 3 : 2;
    static constexpr int kWarps = kTeams * kTeam;
    static constexpr int kThreads = 32 * (kWarps + 1);
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

// transpose of an 8x8 matrix of 16-bit values, lane l holding row l/4, columns 2(l%4), +1
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr uint32_t k64 = 0x64646464u;

// Lane (g = lane/4, t = lane%4).  K values of MMA step j: head values kdim(t, j) + 0..3;
// output tile i: head values vdim(g, i), +1.
template <int D, bool Q8>
__device__ __forceinline__ constexpr int kdim(int t, int j)
{
    return Q8 && D == 128 ? 32 * t + 4 * j : 64 * (j / 4) + 16 * t + 4 * (j % 4);
}
template <int D, bool Q8>
__device__ __forceinline__ constexpr int vdim(int g, int i)
{
    return Q8 && D == 128 ? 16 * g + 2 * i : 64 * (i / 4) + 8 * g + 2 * (i % 4);
}

// ---- one tile of 16 keys ----------------------------------------------------------------
template <int D, bool Q8, int NT>
struct RowState {
    float o[NT][D / 16][4];
    float l[NT][4];      // every key row of the ones-product holds the same sums
    float m[NT][2];      // running maxima of rows 2t, 2t + 1
};

__device__ __forceinline__ bool f16_not_finite(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }

// zeroes the halves of v that are not finite; true where there were some
__device__ __forceinline__ bool drop_not_finite(uint32_t* v)
{
    const bool lo = f16_not_finite(*v), hi = f16_not_finite(*v >> 16);
    if (lo) *v &= 0xffff0000u;
    if (hi) *v &= 0x0000ffffu;
    return lo || hi;
}

// TAIL: the tile reaches past the context, so visibility is tested per key and
// row, and values that are not finite are kept out of the products (0 * NaN
// would reach rows that do not see the key) and added to the rows that do.
template <int D, bool Q8, int NT, bool TAIL>
__device__ __forceinline__ void rows_tile(const uint8_t* blk, int r0, int key0, const uint32_t (&q)[NT][D / 16][2],
                                          float scale_log2, RowState<D, Q8, NT>& st, int ctx, int len,
                                          const uint64_t* row_mask)
{
    using B = KvBlock<D, Q8>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // ---- S^T
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
    const int ra = r0 + g, rb = ra + 8;
    if constexpr (Q8) {
        const __half* const sc = reinterpret_cast<const __half*>(blk + B::kScK);
        constexpr int LD = D / 64;  // 16-byte chunks of a lane per row
        const int sb = D == 128 ? t : t >> 1;
        const __half2 da = __half2half2(sc[ra * (D / 32) + sb]), db = __half2half2(sc[rb * (D / 32) + sb]);
#pragma unroll
        for (int h = 0; h < LD; ++h) {
            const uint4 xa = lds16(blk + B::chunk(ra, LD * t + h)), xb = lds16(blk + B::chunk(rb, LD * t + h));
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
            const int c = 8 * (h >> 1) + 2 * t + (h & 1);
            const uint4 xa = lds16(blk + B::chunk(ra, c)), xb = lds16(blk + B::chunk(rb, c));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16816(s[n], xa.x, xb.x, xa.y, xb.y, q[n][2 * h][0], q[n][2 * h][1]);
                mma16816(s[n], xa.z, xb.z, xa.w, xb.w, q[n][2 * h + 1][0], q[n][2 * h + 1][1]);
            }
        }
    }
    // ---- softmax numerators
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[n][e] *= scale_log2;
            if (TAIL) {
                const int j = key0 + g + (e >> 1) * 8;
                const uint64_t bits = row_mask[8 * n + 2 * t + (e & 1)];
                const bool sees = j < ctx || (j < len && ((bits >> (j - ctx)) & 1));
                if (!sees) s[n][e] = -INFINITY;
            }
        }
        raise |= fmaxf(s[n][0], s[n][2]) > st.m[n][0] + kRaise || fmaxf(s[n][1], s[n][3]) > st.m[n][1] + kRaise;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                const float mn = fmaxf(st.m[n][e], x), f = ex2(st.m[n][e] - mn);
                st.m[n][e] = mn;
                st.l[n][e] *= f;
                st.l[n][e + 2] *= f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    st.o[n][i][e] *= f;
                    st.o[n][i][e + 2] *= f;
                }
            }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float m0 = st.m[n][0] - kShift, m1 = st.m[n][1] - kShift;
        pb[n][0] = transpose8x8(pack_f16(ex2(s[n][0] - m0), ex2(s[n][1] - m1)));
        pb[n][1] = transpose8x8(pack_f16(ex2(s[n][2] - m0), ex2(s[n][3] - m1)));
        constexpr uint32_t one = 0x3c003c00u;
        mma16816(st.l[n], one, one, one, one, pb[n][0], pb[n][1]);
    }
    // ---- O^T: keys 2t, 2t + 1, 2t + 8, 2t + 9 of the tile
    const int k0 = r0 + 2 * t;
    const uint8_t* const vb = blk + B::kVOff;
    bool dropped = false;
    bool in0 = true, in1 = true, in2 = true, in3 = true;  // TAIL: the key is within the sequence
    if (TAIL) {
        const int j = key0 + 2 * t;
        in0 = j < len, in1 = j + 1 < len, in2 = j + 8 < len, in3 = j + 9 < len;
    }
    auto product = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        if (TAIL) {
            const uint32_t m01 = (in0 ? 0xffffu : 0u) | (in1 ? 0xffff0000u : 0u);
            const uint32_t m23 = (in2 ? 0xffffu : 0u) | (in3 ? 0xffff0000u : 0u);
            a0 &= m01, a1 &= m01, a2 &= m23, a3 &= m23;
            dropped |= drop_not_finite(&a0);
            dropped |= drop_not_finite(&a1);
            dropped |= drop_not_finite(&a2);
            dropped |= drop_not_finite(&a3);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(st.o[n][i], a0, a1, a2, a3, pb[n][0], pb[n][1]);
    };
    if constexpr (Q8) {
        const __half* const sc = reinterpret_cast<const __half*>(blk + B::kScK + B::kScBytes);
        const int sb = D == 128 ? g >> 1 : g >> 2;
        constexpr int SL = D / 32;
        const __half2 d01 = __halves2half2(sc[k0 * SL + sb], sc[(k0 + 1) * SL + sb]);
        const __half2 d23 = __halves2half2(sc[(k0 + 8) * SL + sb], sc[(k0 + 9) * SL + sb]);
        constexpr int NW = D / 32;  // words (4 head values) of a lane
        uint32_t v0[NW], v1[NW], v2[NW], v3[NW];
        auto load = [&](int r, uint32_t(&v)[NW]) {
            if constexpr (D == 128) {
                const uint4 x = lds16(vb + B::chunk(r, g));
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(vb + B::chunk(r, g >> 1) + (g & 1) * 8);
                v[0] = x.x, v[1] = x.y;
            }
        };
        load(k0, v0), load(k0 + 1, v1), load(k0 + 8, v2), load(k0 + 9, v3);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const uint32_t pl = __byte_perm(v0[w], v1[w], 0x5140), ph = __byte_perm(v0[w], v1[w], 0x7362);
            const uint32_t rl = __byte_perm(v2[w], v3[w], 0x5140), rh = __byte_perm(v2[w], v3[w], 0x7362);
            product(2 * w, kv_pair(__byte_perm(pl, k64, 0x4140), d01), kv_pair(__byte_perm(pl, k64, 0x4342), d01),
                    kv_pair(__byte_perm(rl, k64, 0x4140), d23), kv_pair(__byte_perm(rl, k64, 0x4342), d23));
            product(2 * w + 1, kv_pair(__byte_perm(ph, k64, 0x4140), d01), kv_pair(__byte_perm(ph, k64, 0x4342), d01),
                    kv_pair(__byte_perm(rh, k64, 0x4140), d23), kv_pair(__byte_perm(rh, k64, 0x4342), d23));
        }
    } else {
#pragma unroll
        for (int pl = 0; pl < D / 64; ++pl) {
            const uint4 x0 = lds16(vb + B::chunk(k0, 8 * pl + g)), x1 = lds16(vb + B::chunk(k0 + 1, 8 * pl + g));
            const uint4 x2 = lds16(vb + B::chunk(k0 + 8, 8 * pl + g)), x3 = lds16(vb + B::chunk(k0 + 9, 8 * pl + g));
            const uint32_t v0[4] = {x0.x, x0.y, x0.z, x0.w}, v1[4] = {x1.x, x1.y, x1.z, x1.w};
            const uint32_t v2[4] = {x2.x, x2.y, x2.z, x2.w}, v3[4] = {x3.x, x3.y, x3.z, x3.w};
#pragma unroll
            for (int w = 0; w < 4; ++w)
                product(4 * pl + w, __byte_perm(v0[w], v1[w], 0x5410), __byte_perm(v0[w], v1[w], 0x7632),
                        __byte_perm(v2[w], v3[w], 0x5410), __byte_perm(v2[w], v3[w], 0x7632));
        }
    }
    if (TAIL && __any_sync(0xffffffffu, dropped)) {
        // rare: whatever its weight, such a value makes the outputs of the rows that see it what it is
        for (int k = 0; k < 16; ++k) {
            const int j = key0 + k;
            if (j >= len) break;
            const int r = r0 + k;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint64_t bits = row_mask[8 * n + 2 * t + e];
                    if (!(j < ctx || ((bits >> (j - ctx)) & 1))) continue;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float v = kv_value<D, Q8>(blk, r, vdim<D, Q8>(g, i) + x, 1);
                            if (!(v - v == 0.0f)) st.o[n][i][e + 2 * x] += v;
                        }
                }
        }
    }
}

// ---- the kernel ----------------------------------------------------------------------------
template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(RowsCfg<NT>::kThreads, 1)
    attn_rows_kernel(const AttnParams p, const int stages, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    using C = RowsCfg<NT>;
    constexpr int RT = C::kRows, kWarps = C::kWarps, kCons = 32 * kWarps;
    extern __shared__ __align__(128) uint8_t sm[];
    uint8_t* const ring = sm;
    float* const merge = reinterpret_cast<float*>(sm + stages * B::kBytes);  // [kTeam][RT][D]
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], seg_full[kSegs], seg_empty[kSegs];
    __shared__ AttnSegment seg_s[kSegs];
    __shared__ uint64_t mask_s[RT];
    __shared__ float m_s[kWarps][RT], l_s[kWarps][RT];
    __shared__ int64_t scratch[kWarps + 1], at_s;
    __shared__ float sum_s[RT];
    __shared__ int seq_s, bad_s[kMaxStages], ok_s[kWarps], seg_bad_s, is_last_s, gone_s;
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kTeam);
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(&seg_full[s], 1);
            mbar_init(&seg_empty[s], kWarps);
        }
        fence_barrier_init();
    }
    const AttnRange rg = attn_range(p, RT, status, scratch, &seq_s, &at_s);  // synchronises the CTA
    if (rg.first >= rg.last) return;

    if (warp == kWarps) {
        // ---- producer
        if (lane == 0) {
            AttnRange w = rg;
            AttnSegment g;
            int64_t at = rg.first;
            const int64_t page_bytes = int64_t(p.c.n_kv_heads) * B::kBytes;
            int it = 0, sg = 0;
            for (; !abort_flag && attn_next(p, RT, &w, &at, &g); ++sg) {
                const int ss = sg % kSegs;
                if (sg >= kSegs && !mbar_wait_bounded(&seg_empty[ss], uint32_t(sg / kSegs - 1) & 1u, p.limit_ns)) {
                    abort_flag = 1;
                    break;
                }
                seg_s[ss] = g;
                mbar_arrive(&seg_full[ss]);
                for (int i = 0; i < g.n; ++i, ++it) {
                    const int s = it % stages;
                    if (it >= stages && !mbar_wait_bounded(&empty[s], uint32_t(it / stages - 1) & 1u, p.limit_ns)) {
                        abort_flag = 1;
                        break;
                    }
                    const int64_t page = kv_page_of(p.c, g.seq, (g.page0 + i) * kKvPage, page_bytes);
                    bad_s[s] = page < 0;
                    if (page < 0) {
                        mbar_arrive(&full[s]);
                        continue;
                    }
                    mbar_arrive_expect_tx(&full[s], B::kBytes);
                    bulk_copy_g2s(ring + s * B::kBytes, p.c.pages + page + int64_t(g.head) * B::kBytes, B::kBytes, &full[s]);
                }
            }
            // copies still in flight land before the CTA can exit
            for (int j = it > stages ? it - stages : 0; j < it; ++j)
                (void)mbar_wait_bounded(&full[j % stages], uint32_t(j / stages) & 1u, p.limit_ns);
        }
        __syncwarp();
        if (abort_flag && lane == 0) atomicOr(status, MQ_DEV_TIMEOUT);
        return;
    }

    // ---- consumers
    const int team = warp / kTeam, wi = warp % kTeam, g8 = lane >> 2, t4 = lane & 3;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait_bounded(bar, parity, p.limit_ns));
        if (!ok) abort_flag = 1;
        return ok;
    };
    int it = 0;
    int64_t done = rg.first;
    for (int sg = 0; done < rg.last; ++sg) {
        const int ss = sg % kSegs;
        bool ok = wait_all(&seg_full[ss], uint32_t(sg / kSegs) & 1u);
        const AttnSegment g = seg_s[ss];
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[ss]);
        const int rows = ok ? min(RT, g.T * p.group - g.row0) : 0, len = g.ctx + g.T;
        RowState<D, Q8, NT> st;
        uint32_t q[NT][D / 16][2];
        if (ok) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = 8 * n + g8, row = g.row0 + r;
                const __half* const src = static_cast<const __half*>(p.a.q) +
                                          int64_t(g.t0 + row / p.group) * p.a.q_ld +
                                          (g.head * p.group + row % p.group) * D;
#pragma unroll
                for (int j = 0; j < D / 16; j += 2) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (r < rows) v = __ldg(reinterpret_cast<const uint4*>(src + kdim<D, Q8>(t4, j)));
                    q[n][j][0] = v.x, q[n][j][1] = v.y, q[n][j + 1][0] = v.z, q[n][j + 1][1] = v.w;
                }
                st.m[n][0] = st.m[n][1] = -3.402823466e38f;  // finite: a row without keys stays at 0 / 0 sums
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    st.l[n][e] = 0.0f;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) st.o[n][i][e] = 0.0f;
                }
            }
        }
        // the rows' masks (the previous segment's readers are past the merge's barriers)
        if (threadIdx.x < RT) {
            uint64_t bits = 0;
            const int node = (g.row0 + int(threadIdx.x)) / p.group;
            if (ok && int(threadIdx.x) < rows) bits = p.a.mask ? __ldg(p.a.mask + g.t0 + node) : ~0ull >> (63 - node);
            mask_s[threadIdx.x] = bits;
        }
        named_barrier_sync(1, kCons);
        bool bad = false;
        for (int i = team; ok && i < g.n; i += C::kTeams) {
            const int n = it + i, s = n % stages;
            ok = wait_all(&full[s], uint32_t(n / stages) & 1u);
            if (!ok) break;
            bad |= bad_s[s] != 0;
            const uint8_t* const blk = ring + s * B::kBytes;
            const int key0 = (g.page0 + i) * kKvPage + 16 * wi;
            if (key0 + 16 <= g.ctx)
                rows_tile<D, Q8, NT, false>(blk, 16 * wi, key0, q, p.scale_log2, st, g.ctx, len, mask_s);
            else if (key0 < len)
                rows_tile<D, Q8, NT, true>(blk, 16 * wi, key0, q, p.scale_log2, st, g.ctx, len, mask_s);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
        it += g.n;
        done += g.n;

        // ---- join the warps: common maxima, then the teams add up in order
        if (g8 == 0)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m_s[warp][8 * n + 2 * t4 + e] = st.m[n][e];
                    l_s[warp][8 * n + 2 * t4 + e] = st.l[n][e];
                }
        if (lane == 0) ok_s[warp] = ok;
        if (threadIdx.x == 0) seg_bad_s = 0, gone_s = 0;
        named_barrier_sync(1, kCons);
        // a wait that ran out in any warp ends all of them here, together
        bool all_ok = true;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all_ok &= ok_s[w] != 0;
        if (!all_ok) break;
        if (bad && lane == 0) seg_bad_s = 1;  // read after the next barrier
        float f[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mm = m_s[0][8 * n + 2 * t4 + e];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, m_s[w][8 * n + 2 * t4 + e]);
                f[n][e] = ex2(st.m[n][e] - mm);
            }
        for (int tm = 0; tm < C::kTeams; ++tm) {
            if (team == tm) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* const row = merge + (wi * RT + 8 * n + 2 * t4 + e) * D;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            float2* const x = reinterpret_cast<float2*>(row + vdim<D, Q8>(g8, i));
                            float2 v = make_float2(st.o[n][i][e] * f[n][e], st.o[n][i][e + 2] * f[n][e]);
                            if (tm) {
                                const float2 y = *x;
                                v.x += y.x, v.y += y.y;
                            }
                            *x = v;
                        }
                    }
            }
            named_barrier_sync(1, kCons);
        }
        const bool seg_bad = seg_bad_s != 0;
        const bool whole = g.n_ctas == 1;
        float* const slot = p.parts + (int64_t(blockIdx.x) * 2 + g.slot) * attn_slot_floats(RT, D);
        for (int x = warp; x < rows * (D / 32); x += kWarps) {
            const int r = x / (D / 32), d = (x % (D / 32)) * 32 + lane;
            float mm = m_s[0][r], sum = 0.0f, v = 0.0f;
            for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, m_s[w][r]);
            for (int w = 0; w < kWarps; ++w) sum += l_s[w][r] * ex2(m_s[w][r] - mm);
            for (int w = 0; w < kTeam; ++w) v += merge[(w * RT + r) * D + d];
            if (whole) {
                if (!seg_bad) attn_emit(p, g, g.row0 + r, D, d - lane, sum == 0.0f ? 0.0f : v / sum);
            } else {
                if (d == 0) {
                    slot[r] = mm;
                    slot[RT + r] = seg_bad ? -1.0f : sum;
                }
                slot[2 * RT + r * D + d] = v;
            }
        }
        if (whole) {
            if (seg_bad && threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
            named_barrier_sync(1, kCons);
            continue;
        }
        named_barrier_sync(1, kCons);
        if (threadIdx.x == 0) is_last_s = attn_arrive(p, g);
        named_barrier_sync(1, kCons);
        if (is_last_s) {
            // ---- the group's last CTA joins its segments, in CTA order
            float* const wgt = merge;  // [n_ctas][RT], free here
            auto slot_of = [&](int c) {
                return p.parts + (int64_t(g.cta0 + c) * 2 + (c == 0 ? g.slot0 : 0)) * attn_slot_floats(RT, D);
            };
            bool gone = false;
            for (int r = warp; r < rows; r += kWarps) {
                float mm = -3.402823466e38f, sum = 0.0f;
                for (int c = lane; c < g.n_ctas; c += 32) mm = fmaxf(mm, __ldcg(slot_of(c) + r));
                for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
                for (int c = lane; c < g.n_ctas; c += 32) {
                    const float f1 = ex2(__ldcg(slot_of(c) + r) - mm), l = __ldcg(slot_of(c) + RT + r);
                    gone |= l < 0.0f;
                    wgt[c * RT + r] = f1;
                    sum += l * f1;
                }
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) sum_s[r] = sum;
            }
            if (gone) gone_s = 1;
            named_barrier_sync(1, kCons);
            if (gone_s) {
                if (threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
            } else {
                for (int x = warp; x < rows * (D / 32); x += kWarps) {
                    const int r = x / (D / 32), d = (x % (D / 32)) * 32 + lane;
                    float v = 0.0f;
#pragma unroll 8
                    for (int c = 0; c < g.n_ctas; ++c)
                        v = fmaf(__ldcg(slot_of(c) + 2 * RT + r * D + d), wgt[c * RT + r], v);
                    attn_emit(p, g, g.row0 + r, D, d - lane, sum_s[r] == 0.0f ? 0.0f : v / sum_s[r]);
                }
            }
        }
        named_barrier_sync(1, kCons);
    }
}

template <int D, bool Q8, int NT>
cudaError_t launch_rows(const AttnParams& p, int grid, int max_smem, unsigned* status, cudaStream_t s)
{
    using B = KvBlock<D, Q8>;
    constexpr int kMerge = kTeam * RowsCfg<NT>::kRows * D * 4;
    int stages = (max_smem - kMerge) / B::kBytes;
    if (stages > kMaxStages) stages = kMaxStages;
    const int smem = stages * B::kBytes + kMerge;
    attn_rows_kernel<D, Q8, NT><<<grid, RowsCfg<NT>::kThreads, smem, s>>>(p, stages, status);
    return cudaGetLastError();
}

template <int NT>
cudaError_t launch_rows_nt(const mq_kv_cache& c, const AttnParams& p, int grid, int max_smem, unsigned* status,
                           cudaStream_t s)
{
    if (c.type == MQ_TYPE_Q8_0)
        return c.head_dim == 128 ? launch_rows<128, true, NT>(p, grid, max_smem, status, s)
                                 : launch_rows<64, true, NT>(p, grid, max_smem, status, s);
    return c.head_dim == 128 ? launch_rows<128, false, NT>(p, grid, max_smem, status, s)
                             : launch_rows<64, false, NT>(p, grid, max_smem, status, s);
}

constexpr int kRowsSmem = 220 * 1024;  // ring and merge buffers; the kernel's static arrays come on top

}  // namespace

// counters of the most groups any call with these heads has, then the partial results
static size_t counters_bytes(const mq_kv_cache& c, int n_heads)
{
    const int rows = n_heads / c.n_kv_heads * MQ_TREE_MAX_TOKENS;
    const size_t groups = size_t(c.n_seqs) * c.n_kv_heads * ((rows + 7) / 8);
    return (groups * 4 + 127) / 128 * 128;
}

size_t attn_workspace_bytes(const mq_kv_cache& c, int n_heads, int max_tokens, int num_sms)
{
    (void)max_tokens;
    return counters_bytes(c, n_heads) + size_t(num_sms) * 2 * attn_slot_floats(16, c.head_dim) * 4;
}

cudaError_t launch_attn(const mq_kv_cache& cache, const mq_attn_args& a, void* ws, int num_sms, unsigned* status,
                        cudaStream_t s)
{
    AttnParams p;
    p.a = a;
    p.c = kv_view(cache);
    p.group = a.n_heads / cache.n_kv_heads;
    p.scale_log2 = float(double(a.scale) * 1.4426950408889634);
    p.counters = static_cast<unsigned*>(ws);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + counters_bytes(cache, a.n_heads));
    p.limit_ns = uint64_t(fault_policy() == FAULT_NONE ? 2000 : 50) * 1000000ull;
    const int rows = p.group * a.max_tokens, RT = rows <= 8 ? 8 : 16;
    // no more CTAs than the bounds allow units
    const int64_t most = int64_t(cache.n_seqs) * ((int64_t(a.max_len) + kKvPage - 1) / kKvPage) * cache.n_kv_heads *
                         ((rows + RT - 1) / RT);
    const int grid = int(most < 1 ? 1 : most < num_sms ? most : num_sms);
    return RT == 8 ? launch_rows_nt<1>(cache, p, grid, kRowsSmem, status, s)
                   : launch_rows_nt<2>(cache, p, grid, kRowsSmem, status, s);
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
    return e;
}

}  // namespace mq
