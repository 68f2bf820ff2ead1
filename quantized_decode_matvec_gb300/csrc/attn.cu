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
__device__ __forceinline__ uint32_t lds16u(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
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

// A lane's places in a tile of the warp's rows r0.. of a block, in bytes from
// the block's start (the rows 8 further have the same permutation, so their
// places are constants away).
template <int D, bool Q8>
struct TilePlaces {
    using B = KvBlock<D, Q8>;
    uint32_t k;       // first 16-byte run of K row r0 + g; the next is at ^ 16 (where there is one)
    uint32_t v0, v1;  // run of V rows r0 + 2t and r0 + 2t + 1
    uint32_t sk, sv;  // q8_0: scales of those K and V rows
    __device__ __forceinline__ TilePlaces(int r0, int g, int t)
    {
        const int ra = r0 + g, rv = r0 + 2 * t;
        if (Q8) {
            k = B::chunk(ra, (D / 64) * t);
            v0 = B::kVOff + B::chunk(rv, D == 128 ? g : g >> 1) + (D == 128 ? 0 : (g & 1) * 8);
            v1 = B::kVOff + B::chunk(rv + 1, D == 128 ? g : g >> 1) + (D == 128 ? 0 : (g & 1) * 8);
            sk = B::kScK + (ra * (D / 32) + (D == 128 ? t : t >> 1)) * 2;
            sv = B::kScK + B::kScBytes + (rv * (D / 32) + (D == 128 ? g >> 1 : g >> 2)) * 2;
        } else {
            k = B::chunk(ra, 2 * t);
            v0 = B::kVOff + B::chunk(rv, g);
            v1 = B::kVOff + B::chunk(rv + 1, g);
            sk = sv = 0;
        }
    }
};

// tail: the tile reaches past the context, so what a row sees is tested key by key
template <int D, bool Q8, int NT>
__device__ __forceinline__ void rows_tile(uint8_t* blk, int r0, int key0, const TilePlaces<D, Q8>& at,
                                          const uint32_t (&q)[NT][D / 16][2], float scale_log2,
                                          RowState<D, Q8, NT>& st, int ctx, int len, const uint64_t* row_mask, bool tail)
{
    using B = KvBlock<D, Q8>;
    constexpr int k8 = 8 * B::kRow;          // eight rows on
    constexpr int s8 = 8 * (D / 32) * 2;     // their scales
    constexpr int kPlane = kKvPage * 128;    // f16: the next 64 values
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t base = smem_u32(blk);
    // ---- S^T
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
    // ---- softmax numerators
    bool raise = false;
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
    if (tail) {
        if (clean_values<D, Q8>(blk, r0, key0, len)) {
#pragma unroll 1
            for (int k = 0; k < min(16, len - key0); ++k) {
                const int j = key0 + k, r = r0 + k;
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
            __syncwarp();
            drop_values<D, Q8>(blk, r0);
        }
        // the next bulk copy into this stage comes after these writes
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }
    auto product = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(st.o[n][i], a0, a1, a2, a3, pb[n][0], pb[n][1]);
    };
    if constexpr (Q8) {
        const uint32_t sv = base + at.sv;
        const uint32_t d01 = __byte_perm(lds16u(sv), lds16u(sv + (D / 32) * 2), 0x5410);
        const uint32_t d23 = __byte_perm(lds16u(sv + s8), lds16u(sv + s8 + (D / 32) * 2), 0x5410);
        constexpr int NW = D / 32;  // words (4 head values) of a lane
        uint32_t v0[NW], v1[NW], v2[NW], v3[NW];
        auto load = [&](uint32_t a, uint32_t(&v)[NW]) {
            if constexpr (D == 128) {
                const uint4 x = lds128(a);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
            } else {
                const uint2 x = lds64(a);
                v[0] = x.x, v[1] = x.y;
            }
        };
        load(base + at.v0, v0), load(base + at.v1, v1), load(base + at.v0 + k8, v2), load(base + at.v1 + k8, v3);
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
            const uint32_t va = base + at.v0 + pl * kPlane, vb = base + at.v1 + pl * kPlane;
            const uint4 x0 = lds128(va), x1 = lds128(vb), x2 = lds128(va + k8), x3 = lds128(vb + k8);
            const uint32_t v0[4] = {x0.x, x0.y, x0.z, x0.w}, v1[4] = {x1.x, x1.y, x1.z, x1.w};
            const uint32_t v2[4] = {x2.x, x2.y, x2.z, x2.w}, v3[4] = {x3.x, x3.y, x3.z, x3.w};
#pragma unroll
            for (int w = 0; w < 4; ++w)
                product(4 * pl + w, __byte_perm(v0[w], v1[w], 0x5410), __byte_perm(v0[w], v1[w], 0x7632),
                        __byte_perm(v2[w], v3[w], 0x5410), __byte_perm(v2[w], v3[w], 0x7632));
        }
    }
}

// ---- the kernel ----------------------------------------------------------------------------
// what the producer hands over with a segment, besides its query rows
struct RowsSegment {
    AttnSegment g;
    int split;  // index among the CTA's groups that it shares with others (at most two), or -1
};

template <int D, bool Q8, int NT>
struct RowsSmem {
    using B = KvBlock<D, Q8>;
    using C = RowsCfg<NT>;
    static constexpr int kQ = C::kRows * D * 2;            // a segment's query rows
    static constexpr int kTile = 32 * 4 + 4;               // floats of one output tile of a warp, padded
    static constexpr int kWarpOut = NT * (D / 16) * kTile; // floats of a warp's outputs
    static constexpr int kFixed = kSegs * kQ + C::kWarps * kWarpOut * 4;
};

template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(RowsCfg<NT>::kThreads, 1)
    attn_rows_kernel(const AttnParams p, const int stages, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    using C = RowsCfg<NT>;
    using S = RowsSmem<D, Q8, NT>;
    constexpr int RT = C::kRows, kWarps = C::kWarps, kCons = 32 * kWarps;
    extern __shared__ __align__(128) uint8_t sm[];
    uint8_t* const ring = sm;
    __half* const q_s = reinterpret_cast<__half*>(sm + stages * B::kBytes);
    float* const out_s = reinterpret_cast<float*>(sm + stages * B::kBytes + kSegs * S::kQ);
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], seg_full[kSegs], seg_empty[kSegs];
    __shared__ __align__(8) uint64_t part_full[2], part_done[2];
    __shared__ RowsSegment seg_s[kSegs];
    __shared__ AttnSegment split_s[2];
    __shared__ uint64_t mask_s[kSegs][RT];
    __shared__ float m_s[kWarps][RT], l_s[kWarps][RT], sum_s[RT];
    __shared__ int2 at_s, scratch[kWarps + 1];
    __shared__ int bad_s[kMaxStages], seen_s[kMaxStages], ok_s[kWarps], pages_bad_s[kWarps], last_s[2], gone_s;
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        gone_s = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kTeam);
            seen_s[s] = 0;
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(&seg_full[s], 1);
            mbar_init(&seg_empty[s], kWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&part_full[s], kWarps);
            mbar_init(&part_done[s], 1);
        }
        fence_barrier_init();
    }
    const AttnRange rg = attn_range(p, RT, status, scratch, &at_s);  // synchronises the CTA
    if (rg.first >= rg.last) return;

    // one outcome for the whole warp
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.limit_ns));
        if (!ok) abort_flag = 1;
        return ok;
    };

    if (warp == kWarps) {
        // ---- producer: lane 0 waits and copies, the warp reads page numbers 32 at a time
        AttnRange w = rg;
        AttnSegment g = {};
        int at = rg.first, it = 0, s = 0, sg = 0, splits = 0;
        uint32_t phase = 0;
        bool ok = true, more = true;
        for (; ok && more; ++sg) {
            more = attn_next(p, RT, &w, &at, &g);
            if (!more) g.n = g.T = 0;
            const int ss = sg % kSegs, rows = more ? min(RT, g.T * p.group - g.row0) : 0;
            const int32_t* const table = p.c.table + int64_t(g.seq) * p.c.table_ld + g.page0;
            int32_t page_l = lane < g.n ? __ldg(table + lane) : 0;
            uint64_t bits = 0;
            const int node = (g.row0 + lane) / p.group;
            if (lane < rows) bits = p.a.mask ? __ldg(p.a.mask + g.t0 + node) : ~0ull >> (63 - node);
            if (sg >= kSegs) ok = wait_all(&seg_empty[ss], uint32_t(sg / kSegs - 1) & 1u);
            if (!ok) break;
            const int split = more && g.n_ctas > 1 ? splits++ : -1;
            if (lane < RT) mask_s[ss][lane] = bits;
            if (lane == 0) {
                seg_s[ss].g = g;
                seg_s[ss].split = split;
                if (split >= 0) split_s[split] = g;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&seg_full[ss], uint32_t(rows) * D * 2);
            __syncwarp();
            if (lane < rows) {
                const int row = g.row0 + lane;
                bulk_copy_g2s(q_s + (ss * RT + lane) * D,
                              static_cast<const __half*>(p.a.q) + int64_t(g.t0 + node) * p.a.q_ld +
                                  (g.head * p.group + row - node * p.group) * D,
                              D * 2, &seg_full[ss]);
            }
            for (int i0 = 0; ok && i0 < g.n; i0 += 32) {
                const int32_t page_now = page_l;
                if (i0 + 32 + lane < g.n) page_l = __ldg(table + i0 + 32 + lane);
                const int m = min(32, g.n - i0);
                for (int i = 0; i < m; ++i, ++it) {
                    const int32_t page = __shfl_sync(0xffffffffu, page_now, i);
                    if (it >= stages) ok = wait_all(&empty[s], phase ^ 1u);
                    if (!ok) break;
                    if (lane == 0) {
                        const bool bad = page < 0 || page >= p.c.n_pages;  // table entries are not trusted
                        bad_s[s] = bad;
                        if (bad) {
                            mbar_arrive(&full[s]);
                        } else {
                            mbar_arrive_expect_tx(&full[s], B::kBytes);
                            bulk_copy_g2s(ring + s * B::kBytes,
                                          p.c.pages + (int64_t(page) * p.c.n_kv_heads + g.head) * B::kBytes, B::kBytes,
                                          &full[s]);
                        }
                    }
                    if (++s == stages) s = 0, phase ^= 1u;
                }
            }
        }
        // the shared groups' arrivals, once the consumers have written their parts
        for (int k = 0; k < splits; ++k) {
            const bool there = mbar_wait_bounded(&part_full[k], 0, p.limit_ns) && !abort_flag;
            if (lane == 0) {
                last_s[k] = there && attn_arrive(p, split_s[k]);
                mbar_arrive(&part_done[k]);
            }
        }
        // copies still in flight land before the CTA can exit
        for (int j = it > stages ? it - stages : 0; j < it; ++j)
            (void)mbar_wait_bounded(&full[j % stages], uint32_t(j / stages) & 1u, p.limit_ns);
        for (int j = sg > kSegs ? sg - kSegs : 0; j < sg; ++j)
            (void)mbar_wait_bounded(&seg_full[j % kSegs], uint32_t(j / kSegs) & 1u, p.limit_ns);
        __syncwarp();
        if (abort_flag && lane == 0) atomicOr(status, MQ_DEV_TIMEOUT);
        return;
    }

    // ---- consumers
    const int team = warp / kTeam, wi = warp % kTeam, g8 = lane >> 2, t4 = lane & 3;
    auto wait_seen = [&](int* word, int value) {
        bool ok = __all_sync(0xffffffffu, load_acquire(word) >= value);
        if (!ok) {
            const uint64_t t0 = global_timer_ns();
            do {
                ok = __all_sync(0xffffffffu, load_acquire(word) >= value);
            } while (__any_sync(0xffffffffu, !ok && global_timer_ns() - t0 < p.limit_ns));
        }
        if (!ok) abort_flag = 1;
        return ok;
    };
    const TilePlaces<D, Q8> places(16 * wi, g8, t4);
    int it = 0, splits = 0;
    bool all_ok = true;
    for (int sg = 0;; ++sg) {
        const int ss = sg % kSegs;
        bool ok = wait_all(&seg_full[ss], uint32_t(sg / kSegs) & 1u);
        const AttnSegment& g = seg_s[ss].g;  // stays until this warp's arrival at seg_empty
        const int ctx = g.ctx, len = ctx + g.T, seg_n = g.n, first_key = g.page0 * kKvPage + 16 * wi;
        RowState<D, Q8, NT> st;
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
            st.m[n][0] = st.m[n][1] = -3.402823466e38f;  // finite: a row without keys keeps zero sums
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                st.l[n][e] = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) st.o[n][i][e] = 0.0f;
            }
        }
        bool bad = false;
        int s = (it + team) % stages;
        uint32_t phase = uint32_t((it + team) / stages) & 1u;
#pragma unroll 1
        for (int i = team; ok && i < seg_n; i += C::kTeams) {
            const int n = it + i;
            // The stage's previous use was another team's page, which may not even have
            // landed; a wait by parity tells two successive uses apart only, so that team's
            // word that it has comes first.
            ok = n < stages || wait_seen(&seen_s[s], n - stages + 1);
            ok = ok && wait_all(&full[s], phase);
            if (ok && wi == 0 && lane == 0) store_release(&seen_s[s], n + 1);
            if (!ok) break;
            bad |= bad_s[s] != 0;
            uint8_t* const blk = ring + s * B::kBytes;
            const int key0 = first_key + i * kKvPage;
            if (key0 < len)
                rows_tile<D, Q8, NT>(blk, 16 * wi, key0, places, q, p.scale_log2, st, ctx, len, mask_s[ss], key0 + 16 > ctx);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            s += C::kTeams;
            if (s >= stages) s -= stages, phase ^= 1u;
        }
        it += seg_n;

        // ---- join the warps that had pages: each leaves its tiles as it holds them
        float* const mine = out_s + warp * S::kWarpOut;
        if (team < seg_n) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float4*>(mine + (n * (D / 16) + i) * S::kTile + 4 * lane) =
                        make_float4(st.o[n][i][0], st.o[n][i][1], st.o[n][i][2], st.o[n][i][3]);
        }
        if (g8 == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m_s[warp][8 * n + 2 * t4 + e] = st.m[n][e];
                    l_s[warp][8 * n + 2 * t4 + e] = st.l[n][e];
                }
        }
        if (lane == 0) ok_s[warp] = ok, pages_bad_s[warp] = bad;
        named_barrier_sync(1, kCons);
        // a wait that ran out in any warp ends all of them here, together
        const int flags = lane < kWarps ? (ok_s[lane] ? 0 : 1) | (pages_bad_s[lane] ? 2 : 0) : 0;
        all_ok = !__any_sync(0xffffffffu, flags & 1);
        const bool seg_bad = __any_sync(0xffffffffu, flags & 2);
        if (!all_ok || seg_n == 0) break;  // failed, or the end
        const int split = seg_s[ss].split, rows = min(RT, g.T * p.group - g.row0);
        const int nw = min(C::kTeams, seg_n) * kTeam;  // warps that had pages
        float* const slot = p.parts + (int64_t(blockIdx.x) * 2 + g.slot) * attn_slot_floats(RT, D);
#pragma unroll 1
        for (int x = warp; x < rows * (D / 32); x += kWarps) {
            const int r = x / (D / 32), d = (x % (D / 32)) * 32 + lane;
            // lane w: warp w's maximum and weight
            const float mw = lane < nw ? m_s[lane][r] : -3.402823466e38f;
            float mm = mw;
#pragma unroll
            for (int o = 8; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
            const float fw = ex2(mw - mm);
            float sum = lane < nw ? l_s[lane][r] * fw : 0.0f;
#pragma unroll
            for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            mm = __shfl_sync(0xffffffffu, mm, 0);
            sum = __shfl_sync(0xffffffffu, sum, 0);
            // value d of row r in a warp's tiles
            const int g_of = Q8 && D == 128 ? d / 16 : (d % 64) / 8;
            const int i_of = Q8 && D == 128 ? (d % 16) / 2 : 4 * (d / 64) + (d % 8) / 2;
            const float* const src = out_s + ((r / 8) * (D / 16) + i_of) * S::kTile +
                                     4 * (4 * g_of + (r % 8) / 2) + (r & 1) + 2 * (d & 1);
            float v = 0.0f;
#pragma unroll 4
            for (int w = 0; w < nw; ++w) v = fmaf(src[w * S::kWarpOut], __shfl_sync(0xffffffffu, fw, w), v);
            if (split < 0) {
                if (!seg_bad) attn_emit(p, g, g.row0 + r, D, d - lane, sum == 0.0f ? 0.0f : v / sum);
            } else {
                if (d == 0) {
                    slot[r] = mm;
                    slot[RT + r] = seg_bad ? -1.0f : sum;
                }
                slot[2 * RT + r * D + d] = v;
            }
        }
        __syncwarp();
        if (lane == 0) {
            if (split >= 0) mbar_arrive(&part_full[split]);
            mbar_arrive(&seg_empty[ss]);
        }
        if (split < 0 && seg_bad && threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        splits += split >= 0;
        named_barrier_sync(1, kCons);  // out_s, m_s, l_s are free again
    }
    if (!all_ok) {
        if (lane == 0)
            for (int k = splits; k < 2; ++k) mbar_arrive(&part_full[k]);  // the producer finds abort_flag set
        return;
    }

    // ---- the shared groups whose last CTA this is: their segments joined in CTA order
    if (splits > 0) {
        bool ok = true;
        for (int k = 0; k < splits; ++k) ok = wait_all(&part_done[k], 0) && ok;
        if (lane == 0) ok_s[warp] = ok;
        named_barrier_sync(1, kCons);
        if (__any_sync(0xffffffffu, lane < kWarps && !ok_s[lane])) return;
    }
    for (int k = 0; k < splits; ++k) {
        if (!last_s[k]) continue;
        const AttnSegment& g = split_s[k];
        const int rows = min(RT, g.T * p.group - g.row0);
        float* const wgt = reinterpret_cast<float*>(ring);  // [n_ctas][RT]; every copy has landed and been read
        auto slot_of = [&](int c) {
            return p.parts + (int64_t(g.cta0 + c) * 2 + (c == 0 ? g.slot0 : 0)) * attn_slot_floats(RT, D);
        };
        bool gone = false;
        for (int r = warp; r < RT; r += kWarps) {
            float mm = -3.402823466e38f, sum = 0.0f;
            if (r < rows) {
                for (int c = lane; c < g.n_ctas; c += 32) mm = fmaxf(mm, __ldcg(slot_of(c) + r));
#pragma unroll
                for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
            }
            for (int c = lane; c < g.n_ctas; c += 32) {
                float f1 = 0.0f;
                if (r < rows) {
                    const float l = __ldcg(slot_of(c) + RT + r);
                    f1 = ex2(__ldcg(slot_of(c) + r) - mm);
                    gone |= l < 0.0f;
                    sum = fmaf(l, f1, sum);
                }
                wgt[c * RT + r] = f1;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) sum_s[r] = sum;
        }
        if (gone) gone_s = 1 + k;
        named_barrier_sync(1, kCons);
        if (gone_s == 1 + k) {
            if (threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
            continue;
        }
        // warp w adds up CTAs w, w + kWarps, ...; a lane holds four values of each 128 of the rows
        constexpr int NV = RT * D / 128;
        float4 acc[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c = warp; c < g.n_ctas; c += kWarps) {
            const float4* const src = reinterpret_cast<const float4*>(slot_of(c) + 2 * RT) + lane;
            float4 x[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v)
                x[v] = (v * 128 + lane * 4) / D < rows ? __ldcg(src + v * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const float f1 = wgt[c * RT + (v * 128 + lane * 4) / D];
                acc[v].x = fmaf(x[v].x, f1, acc[v].x);
                acc[v].y = fmaf(x[v].y, f1, acc[v].y);
                acc[v].z = fmaf(x[v].z, f1, acc[v].z);
                acc[v].w = fmaf(x[v].w, f1, acc[v].w);
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            *reinterpret_cast<float4*>(out_s + warp * RT * D + v * 128 + lane * 4) = acc[v];
        named_barrier_sync(1, kCons);
        for (int x = warp; x < rows * (D / 32); x += kWarps) {
            const int r = x / (D / 32), d = (x % (D / 32)) * 32 + lane;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += out_s[(w * RT + r) * D + d];
            attn_emit(p, g, g.row0 + r, D, d - lane, sum_s[r] == 0.0f ? 0.0f : v / sum_s[r]);
        }
        named_barrier_sync(1, kCons);
    }
}

constexpr int kRowsSmem = 222 * 1024;  // ring and merge buffers; the kernel's static arrays come on top

template <int D, bool Q8, int NT>
cudaError_t launch_rows(const AttnParams& p, int grid, int max_smem, unsigned* status, cudaStream_t s)
{
    using B = KvBlock<D, Q8>;
    using S = RowsSmem<D, Q8, NT>;
    int stages = (max_smem - S::kFixed) / B::kBytes;
    if (stages > kMaxStages) stages = kMaxStages;
    static_assert((kRowsSmem - S::kFixed) / B::kBytes >= RowsCfg<NT>::kTeams, "each team needs a page to work on");
    const int smem = stages * B::kBytes + S::kFixed;
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
