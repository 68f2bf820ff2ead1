// attn_tc.cu -- attention of many query rows per key/value head (trees of more
// than a few tokens) over the paged cache, on the tensor cores.
//
// The same sums as attn.cu; with dozens to hundreds of query rows per
// key/value head every cached byte is used that often, and the products and
// the exponentials bound it instead of the cache's bytes.  Per CTA (one per
// SM, an equal share of all pages, mq_attn.cuh), in steps of two pages:
//   warps 0-3, 4-7  softmax of two tiles of 128 query rows, a thread per row
//   warps 8-11      the operands: q8_0 codes to f16 in the tensor cores'
//                   layout; both types: the values of pages that reach past
//                   the context made finite
//   warp 12         segments, and bulk copies in the order of use: q8_0 into a
//                   ring of half blocks, f16 into the operands themselves
//   warp 13         tensor memory and the MMAs
// Tensor memory holds for each tile the scores of a step (128 columns), in
// their place the probabilities (f16, the A operand of the second product),
// and the fp32 outputs:
//   S[128][128] = Q K^T       Q and K from shared memory, K-major
//   O[128][D] += P V          V from shared memory as it lies, MN-major
// Steps of 128 keys because an MMA of N = 64 takes as long as one of 128 (66
// cycles measured).  While one tile's probabilities are formed the other
// tile's products run: the issue order is
//   S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...
// and a step's second product starts when the first half of its probabilities
// is there.  With more than 128 rows the tiles are the rows' halves and both
// take every step; with fewer both hold the same rows, take the steps in turn
// and are joined at the end.
// Probabilities are 2^(s - m + 7) in f16, m the row's running maximum, which is
// raised (and O rescaled in tensor memory) only when a score passes it by more
// than 8, so they stay below 2^15; a key at 2^-21 of the largest is still a
// normal number.  Scores, maxima, sums and outputs are fp32.
// f16 is what the second product takes at full rate beside f16 values, and it
// halves the probabilities' columns; each is rounded to nearest, 2^-11, as the
// output is.  Their sum is of the unrounded numbers: of the rounded ones it
// would take 128 conversions more per row and step, in the warps that a tile's
// products wait for, to take out the roundings' mean, which many keys leave
// small.  Root mean square error of the case below against 64 bits, relative:
// 2.9e-4, where a result that is only rounded once has 2.1e-4.
//
// Measured (28 query heads on 4 of 128, q8_0): four trees of 64 nodes over 8190
// to 32700 tokens 77 us, 720 TFLOP/s, 0.38 of the dense f16 rate.  The tensor
// pipe is busy 38 % of the time: a step's probabilities stand between its two
// products, and of the time per tile and step (about 1800 cycles; the MMAs take
// 1056) the rest is waiting for them, for operands, and the commits.  Start, the
// segments' ends and the join take about 15 us of a call.
#include "mq_attn.cuh"
#include "mq_umma.cuh"

namespace mq {

namespace {

constexpr int kTcRows = 256;  // query rows of a block
constexpr int kTcSegs = 4;
constexpr int kStep = 2 * kKvPage;  // keys
constexpr int kConv = 4;  // operand warps
constexpr int kConvThreads = 32 * kConv;
constexpr int kWarpSeg = 8 + kConv, kWarpMma = kWarpSeg + 1;
constexpr int kTcThreads = 32 * (kWarpMma + 1);
constexpr float kTcRaise = 8.0f, kTcShift = 7.0f, kLowest = -3.402823466e38f;
constexpr uint32_t kColO = 0, kColS = 256;  // tensor memory columns of tile 0; of tile 1 128 further

// Shared memory: a 128-row operand tile is D/64 planes of [128 rows][64 f16], each with the 128-byte swizzle.  K and V
// tiles of a step pass through one ring, in the order of their use; q8_0 comes through a ring of units before, each
// the codes and scales of the keys or values of a step's two pages.
template <int D, bool Q8>
struct TcCfg {
    static constexpr int kPlane = 128 * 128;
    static constexpr int kTile = D / 64 * kPlane;
    static constexpr int kOps = D == 128 ? (Q8 ? 3 : 4) : 6;
    static constexpr int kCodes = kKvPage * D, kHalf = kCodes + KvBlock<D, true>::kScBytes;  // of a page
    static constexpr int kUnit = 2 * kHalf, kUnits = !Q8 ? 0 : D == 128 ? 3 : 6;
    static constexpr int kSmem = 1024 + 2 * kTile + kOps * kTile + kUnits * kUnit;
};
// byte of 16-byte chunk c of row r of an operand tile
__device__ __forceinline__ int tc_chunk(int r, int c)
{
    return (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// The order of a segment's 2n tiles, by position: K(0) V(0) K(1) V(1) .. where both tiles of rows take every step, and
// where they take the steps in turn the scores are a step further ahead: K(0) K(1) V(0) K(2) V(1) .. V(n-1).
struct TcTile {
    int is_v, step;
};
__device__ __forceinline__ TcTile tc_tile_at(int pos, int n, bool halves)
{
    if (halves) return TcTile{pos & 1, pos >> 1};
    if (pos == 0) return TcTile{0, 0};
    if (pos == 2 * n - 1) return TcTile{1, n - 1};
    return pos & 1 ? TcTile{0, (pos + 1) >> 1} : TcTile{1, (pos - 2) >> 1};
}
__device__ __forceinline__ int tc_pos_k(int st, bool halves) { return halves ? 2 * st : st == 0 ? 0 : 2 * st - 1; }
__device__ __forceinline__ int tc_pos_v(int st, int n, bool halves)
{
    return halves ? 2 * st + 1 : st == n - 1 ? 2 * n - 1 : 2 * st + 2;
}

struct TcSegment {
    AttnSegment g;
    int odd, bad;  // a value that is not finite was dropped; a page outside the cache
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// true in one lane of the warp, always the same one
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem], one MMA of M x N x 16 (issued by one thread)
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// descriptor of an MN-major tile with the 128-byte swizzle: rows of 64 values (one per K index), eight rows of K
// 1024 bytes apart, the next 64 values of N `plane` bytes on
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t smem_addr, uint32_t plane)
{
    uint64_t d = 0;
    d |= uint64_t((smem_addr >> 4) & 0x3FFFu);
    d |= uint64_t(plane >> 4) << 16;
    d |= uint64_t(1024u >> 4) << 32;
    d |= uint64_t(1u) << 46;
    d |= uint64_t(2u) << 61;
    return d;
}
constexpr uint32_t kBMajorMn = 1u << 16;  // instruction descriptor: B is MN-major

// exponent bits all ones in either half (they carry into the sign's place)
__device__ __forceinline__ bool pair_not_finite(uint32_t v)
{
    return (((v & 0x7c007c00u) + 0x04000400u) & 0x80008000u) != 0;
}
__device__ __forceinline__ uint32_t drop_pair(uint32_t v)
{
    if ((v & 0x7c00u) == 0x7c00u) v &= 0xffff0000u;
    if ((v & 0x7c000000u) == 0x7c000000u) v &= 0x0000ffffu;
    return v;
}

// ---- operands (warps 8-11, thread x of 128): 64 rows from row0 on of a tile ----------------------
// The loops that every page passes are kept short: with all their rare cases in line they and the
// softmax's outgrew the instruction cache, and warps waited for instructions 40 % of the time.

// q8_0 codes and scales of a unit, both pages or (pages = 1) the first
template <int D>
__device__ __forceinline__ void tc_convert(const uint8_t* unit, uint8_t* tile, int pages, int x)
{
    using R = KvBlock<D, true>;
    using C = TcCfg<D, true>;
    constexpr int N = D / 32;  // 16-byte chunks of codes per thread and page, loaded a page ahead of their use
    const int r0 = x / (D / 16), c = x % (D / 16);
    uint4 in[2][N];
    uint32_t d[2][N];
    auto load = [&](int h) {
        const uint8_t* const u = unit + h * C::kHalf;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = i * (kConvThreads / (D / 16)) + r0;
            in[h][i] = lds16(u + R::chunk(r, c));
            d[h][i] = *reinterpret_cast<const uint16_t*>(u + C::kCodes + (r * (D / 32) + (c >> 1)) * 2) * 0x10001u;
        }
    };
    // a chunk of codes is two of f16; the lanes of the second plane store theirs in the other order: no bank twice
    const bool swap = (c & 4) != 0;
    const int c0 = 2 * c + swap;
    load(0);
    if (pages > 1) load(1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h >= pages) break;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = h * kKvPage + i * (kConvThreads / (D / 16)) + r0;
            const uint4 v = in[h][i];
            const uint32_t w[4] = {swap ? v.z : v.x, swap ? v.w : v.y, swap ? v.x : v.z, swap ? v.y : v.w};
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u[2 * k] = kv_pair(__byte_perm(w[k], 0x64646464u, 0x4140), d[h][i]);
                u[2 * k + 1] = kv_pair(__byte_perm(w[k], 0x64646464u, 0x4342), d[h][i]);
            }
            *reinterpret_cast<uint4*>(tile + tc_chunk(r, c0)) = make_uint4(u[0], u[1], u[2], u[3]);
            *reinterpret_cast<uint4*>(tile + tc_chunk(r, c0 ^ 1)) = make_uint4(u[4], u[5], u[6], u[7]);
        }
    }
}
// values of a page that reaches past the context: rows past the sequence zeroed, what is not finite dropped (true)
template <int D>
__device__ __noinline__ bool tc_clean(uint8_t* tile, int row0, int key0, int len, int x)
{
    bool odd = false;
    for (int i = x; i < kKvPage * (D / 8); i += kConvThreads) {
        const int r = i / (D / 8);
        uint4* const v = reinterpret_cast<uint4*>(tile + tc_chunk(row0 + r, i % (D / 8)));
        if (key0 + r >= len) {
            *v = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint4 y = *v;
        if (pair_not_finite(y.x) || pair_not_finite(y.y) || pair_not_finite(y.z) || pair_not_finite(y.w)) {
            odd = true;
            y.x = drop_pair(y.x), y.y = drop_pair(y.y), y.z = drop_pair(y.z), y.w = drop_pair(y.w);
            *v = y;
        }
    }
    return odd;
}
// zeros
template <int D>
__device__ __noinline__ void tc_zero(uint8_t* tile, int row0, int x)
{
    for (int i = x; i < kKvPage * (D / 8); i += kConvThreads)
        *reinterpret_cast<uint4*>(tile + tc_chunk(row0 + i / (D / 8), i % (D / 8))) = make_uint4(0, 0, 0, 0);
}

// A row's outputs d0 .. d0 + 31 are written (to slot, or where tc_emit puts them): what was dropped because it is
// not finite, and the row sees, makes an output what it is (of a q8_0 block, its scale).
template <int D, bool Q8>
__device__ __noinline__ void tc_add_dropped(const AttnParams& p, const AttnSegment& g, int row, uint64_t mask, int d0,
                                            float* slot)
{
    const int node = attn_row_token(p, row), h = (g.head - node) * p.group + row;
    const int64_t tok = g.t0 + node;
    for (int d = d0; d < d0 + 32; ++d) {
        float add = 0.0f;
        for (int pg = max(g.page0, g.ctx / kKvPage); pg < g.page0 + g.n; ++pg) {
            const int64_t page = kv_page_of(p.c, g.seq, pg * kKvPage, int64_t(p.c.n_kv_heads) * KvBlock<D, Q8>::kBytes);
            if (page < 0) continue;
            const uint8_t* const blk = p.c.pages + page + int64_t(g.head) * KvBlock<D, Q8>::kBytes;
            for (int r = 0; r < kKvPage; ++r) {
                const int j = pg * kKvPage + r;
                if (j >= g.ctx + g.T || (j >= g.ctx && !((mask >> (j - g.ctx)) & 1))) continue;
                const float v = kv_value<D, Q8>(blk, r, d, 1);
                if (!(v - v == 0.0f)) add += v;
            }
        }
        if (add == 0.0f) continue;
        if (slot) {
            slot[2 * kTcRows + (d / 4 * kTcRows + row - g.row0) * 4 + d % 4] += add;
        } else if (p.a.out_type == MQ_TYPE_F16) {
            __half* const o = static_cast<__half*>(p.a.out) + tok * p.a.out_ld + h * D + d;
            *o = __float2half_rn(__half2float(*o) + add);
        } else {
            *reinterpret_cast<__half*>(static_cast<uint8_t*>(p.a.out) +
                                       (tok * (p.a.n_heads * D / 32) + (h * D + d) / 32) * kQ8Bytes) = __float2half_rn(add);
        }
    }
}

// 32 outputs d0.. of a row, by one thread
__device__ __forceinline__ void tc_emit(const AttnParams& p, const AttnSegment& g, int row, int D, int d0,
                                        const float (&o)[32], float inv)
{
    const int node = attn_row_token(p, row), h = (g.head - node) * p.group + row;
    const int64_t tok = g.t0 + node;
    if (p.a.out_type == MQ_TYPE_F16) {
        uint4* const dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.a.out) + tok * p.a.out_ld + h * D + d0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_f16(o[8 * i] * inv, o[8 * i + 1] * inv), pack_f16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                pack_f16(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                pack_f16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
    } else {
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(fabsf(o[i] * inv)));
        const Q8Scale s = q8_scale_of(__uint_as_float(top));
        uint16_t* const dst = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.a.out) +
                                                          (tok * (p.a.n_heads * D / 32) + (h * D + d0) / 32) * kQ8Bytes);
        dst[0] = __half_as_ushort(__float2half_rn(s.d));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            int a, b;
            if (!q8_code_fast(o[2 * i] * inv, s, &a)) a = q8_code_exact(o[2 * i] * inv, s.d);
            if (!q8_code_fast(o[2 * i + 1] * inv, s, &b)) b = q8_code_exact(o[2 * i + 1] * inv, s.d);
            dst[1 + i] = uint16_t((a & 255) | (b & 255) << 8);
        }
    }
}

// ---- the kernel --------------------------------------------------------------------------------
template <int D, bool Q8>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const AttnParams p, unsigned* status)
{
    using C = TcCfg<D, Q8>;
    using B = KvBlock<D, Q8>;
    constexpr int kOps = C::kOps, kUnits = Q8 ? C::kUnits : 1;
    extern __shared__ uint8_t sm_raw[];
    __shared__ __align__(8) uint64_t unit_full[kUnits], unit_free[kUnits], op_full[kOps], op_ready[kOps], op_free[kOps];
    __shared__ int op_bad[Q8 ? kUnits : kOps];  // bit h: the step's page h is not in the cache, so not copied
    __shared__ __align__(8) uint64_t q_ready[2], s_ready[2], p_ready[2][2], o_done[2], seg_full[kTcSegs], seg_empty[kTcSegs];
    __shared__ __align__(8) uint64_t tile_done;  // the converters' stores to a tile that one of them corrects
    __shared__ __align__(8) uint64_t mma_done;   // all that was issued
    __shared__ TcSegment seg_s[kTcSegs];
    __shared__ float join_m[2][128], join_l[2][128];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the swizzled tiles want 1024-byte alignment
    uint8_t* const sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    uint8_t* const q_s = sm;
    uint8_t* const op_s = sm + 2 * C::kTile;
    uint8_t* const unit_s = op_s + kOps * C::kTile;
    float* const join = reinterpret_cast<float*>(q_s + C::kTile);  // [32][128]; tile 1's queries are not used then

    if (threadIdx.x < kOps) {
        mbar_init(&op_full[threadIdx.x], 1);
        mbar_init(&op_ready[threadIdx.x], kConv);
        mbar_init(&op_free[threadIdx.x], 1);
    } else if (threadIdx.x >= 32 && threadIdx.x < 32 + kUnits) {
        mbar_init(&unit_full[threadIdx.x - 32], 1);
        mbar_init(&unit_free[threadIdx.x - 32], kConv);
    } else if (threadIdx.x >= 64 && threadIdx.x < 66) {
        const int k = threadIdx.x - 64;
        mbar_init(&q_ready[k], 4);
        mbar_init(&s_ready[k], 1);
        mbar_init(&p_ready[k][0], 4);
        mbar_init(&p_ready[k][1], 4);
        mbar_init(&o_done[k], 1);
    } else if (threadIdx.x >= 96 && threadIdx.x < 96 + kTcSegs) {
        mbar_init(&seg_full[threadIdx.x - 96], 1);
        mbar_init(&seg_empty[threadIdx.x - 96], 8 + kConv + 1);  // softmax and operand warps, the MMA warp
        if (threadIdx.x == 96) {
            mbar_init(&tile_done, kConv);
            mbar_init(&mma_done, 1);
            abort_flag = 0;
        }
    }
    fence_barrier_init();
    griddep_launch_dependents();  // the join may take its place; it waits for this grid's end
    AttnRange w;
    if (warp == kWarpSeg) w = attn_range(p, kTcRows, status);
    if (warp == kWarpMma) tmem_alloc(&tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    // one outcome for the whole warp
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait_bounded(bar, parity, p.limit_ns));
        if (!ok) abort_flag = 1;
        return ok;
    };

    if (warp == kWarpSeg) {
        // ---- segments and copies; lane h: page h of a step
        AttnSegment g = {};
        int at = w.first, sg = 0, k = 0;  // k: tiles before
        bool ok = true, more = true;
        int4 start[2] = {};  // the last segment's group, if it starts here and others go on with it
        for (; ok && more; ++sg) {
            more = attn_next(p, kTcRows, &w, &at, &g);
            if (!more) g.n = g.T = 0;
            if (more && g.n_ctas > 1 && g.cta0 == int(blockIdx.x)) attn_shared(g, start);
            const int ss = sg % kTcSegs;
            if (sg >= kTcSegs) ok = wait_all(&seg_empty[ss], uint32_t(sg / kTcSegs - 1) & 1u);
            if (!ok) break;
            if (lane == 0) {
                seg_s[ss].g = g;
                seg_s[ss].odd = seg_s[ss].bad = 0;
                mbar_arrive(&seg_full[ss]);
            }
            __syncwarp();
            const int32_t* const table = p.c.table + int64_t(g.seq) * p.c.table_ld + g.page0;
            const int n = (g.n + 1) / 2;
            const bool halves = g.T * p.group - g.row0 > 128;
            for (int pos = 0; ok && pos < 2 * n; ++pos, ++k) {
                const TcTile tl = tc_tile_at(pos, n, halves);
                const int i = 2 * tl.step + (lane & 1), pages = min(2, g.n - 2 * tl.step);
                const int64_t page = i < g.n ? __ldg(table + i) : -1;
                const bool there = page >= 0 && page < p.c.n_pages;  // table entries are not trusted
                const unsigned both = __ballot_sync(0xffffffffu, there) & 3u;
                const uint8_t* const src = p.c.pages + (there ? (page * p.c.n_kv_heads + g.head) * B::kBytes : 0);
                const bool withheld = p.withhold && sg == 0 && pos == 2 * n - 1;  // test-only fault
                // q8_0: the next unit; f16: the tile itself
                const int b = k % (Q8 ? kUnits : kOps);
                uint64_t* const full = Q8 ? &unit_full[b] : &op_full[b];
                if (k >= (Q8 ? kUnits : kOps))
                    ok = wait_all(Q8 ? &unit_free[b] : &op_free[b], uint32_t(k / (Q8 ? kUnits : kOps) - 1) & 1u);
                if (!ok) break;
                if (lane == 0 && !withheld) {
                    op_bad[b] = int(~both & (pages == 2 ? 3u : 1u));
                    if (both)
                        mbar_arrive_expect_tx(full, uint32_t(__popc(both)) * (Q8 ? C::kHalf : kKvPage * D * 2));
                    else
                        mbar_arrive(full);
                }
                __syncwarp();
                if (lane < 2 && there && !withheld) {
                    if (Q8) {
                        uint8_t* const dst = unit_s + b * C::kUnit + lane * C::kHalf;
                        bulk_copy_g2s(dst, src + (tl.is_v ? B::kVOff : 0), C::kCodes, full);
                        bulk_copy_g2s(dst + C::kCodes, src + B::kScK + (tl.is_v ? B::kScBytes : 0), B::kScBytes, full);
                    } else {
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            bulk_copy_g2s(op_s + b * C::kTile + x * C::kPlane + lane * (kKvPage * 128),
                                          src + (tl.is_v ? B::kVOff : 0) + x * (kKvPage * 128), kKvPage * 128, full);
                    }
                }
            }
        }
        // every CTA says so in every call, one that gave up too: the join finds nothing of another call
        if (lane < 2) p.shared[2 * blockIdx.x + lane] = lane == 0 ? start[0] : start[1];
        // copies still in flight land before the CTA can exit
        constexpr int kRing = Q8 ? kUnits : kOps;
        for (int j = k > kRing ? k - kRing : 0; j < k; ++j)
            (void)mbar_wait_bounded(Q8 ? &unit_full[j % kRing] : &op_full[j % kRing], uint32_t(j / kRing) & 1u, p.limit_ns);
    } else if (warp >= 8 && warp < kWarpSeg) {
        // ---- operands, tile by tile
        const int x = threadIdx.x - 256;
        int k = 0;  // tiles before
        uint32_t done_ph = 0;
        bool ok = true;
        for (int sg = 0; ok; ++sg) {
            const int ss = sg % kTcSegs;
            ok = wait_all(&seg_full[ss], uint32_t(sg / kTcSegs) & 1u);
            if (!ok) break;
            const AttnSegment& g = seg_s[ss].g;
            const int n = (g.n + 1) / 2, gn = g.n, key_base = g.page0 * kKvPage, ctx = g.ctx, len = g.ctx + g.T;
            const bool halves = g.T * p.group - g.row0 > 128;
            if (n == 0) break;
            for (int pos = 0; pos < 2 * n; ++pos, ++k) {
                const TcTile tl = tc_tile_at(pos, n, halves);
                const int b = k % kOps;
                uint8_t* const tile = op_s + b * C::kTile;
                const int s = k % kUnits;
                if (Q8) {
                    ok = wait_all(&unit_full[s], uint32_t(k / kUnits) & 1u);
                    ok = ok && (k < kOps || wait_all(&op_free[b], uint32_t(k / kOps - 1) & 1u));
                } else {
                    ok = wait_all(&op_full[b], uint32_t(k / kOps) & 1u);
                }
                if (!ok) break;
                const int bad = op_bad[Q8 ? s : b], pages = min(2, gn - 2 * tl.step);
                if (Q8) {
                    tc_convert<D>(unit_s + s * C::kUnit, tile, pages, x);  // of a page that is not there, whatever it is
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&unit_free[s]);
                }
                bool odd = false;
                const int key0 = key_base + tl.step * kStep;
                if (tl.is_v && (bad || pages < 2 || key0 + kStep > ctx)) {
                    if (Q8) {  // the rows that other warps stored; a warp that gave up does not come
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tile_done);
                        ok = wait_all(&tile_done, done_ph);
                        done_ph ^= 1u;
                        if (!ok) break;
                    }
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        // such values weigh nothing, but they are multiplied with the weight 0
                        if (h >= pages || (bad >> h & 1))
                            tc_zero<D>(tile, h * kKvPage, x);
                        else if (key0 + (h + 1) * kKvPage > ctx)
                            odd |= tc_clean<D>(tile, h * kKvPage, key0 + h * kKvPage, len, x);
                    }
                }
                if (odd) seg_s[ss].odd = 1;
                if (bad && lane == 0) seg_s[ss].bad = 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&op_ready[b]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[ss]);
        }
    } else if (warp == kWarpMma) {
        // ---- MMA issuer.  The whole warp goes through the loops with values that the compiler knows to be the same
        // in all lanes, and one lane issues: with the loops in one lane's branch every operand went through a vector
        // register, and an MMA of 66 cycles took 92 to issue.
        constexpr uint32_t idesc_s = umma_idesc_f16_f32(128, kStep);
        constexpr uint32_t idesc_o = umma_idesc_f16_f32(128, D) | kBMajorMn;
        const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
        // tile 0 of the queries, operand 0 as K and as V; an address within or in another is added to the
        // descriptor's address field
        const uint64_t q_d = umma_desc_sw128(smem_u32(q_s)), k_d = umma_desc_sw128(smem_u32(op_s)),
                       v_d = umma_desc_mn(smem_u32(op_s), C::kPlane);
        int it = 0;  // tiles before this segment
        uint32_t pph[2] = {0, 0}, qph = 0;  // phases of p_ready and q_ready
        bool ok = true;
        for (int sg = 0; ok; ++sg) {
            const int ss = sg % kTcSegs;
            ok = wait_all(&seg_full[ss], uint32_t(sg / kTcSegs) & 1u);
            if (!ok) break;
            const int n = __reduce_max_sync(0xffffffffu, (seg_s[ss].g.n + 1) / 2);  // steps
            if (n == 0) break;
            const bool halves = __reduce_max_sync(0xffffffffu, seg_s[ss].g.T * p.group - seg_s[ss].g.row0) > 128;
            const int items = halves ? 2 * n : n;
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[ss]);
            ok = wait_all(&q_ready[0], qph) && wait_all(&q_ready[1], qph);
            qph ^= 1u;
            // K of item j's step is there, where item j is the first to use it, and so is what `bar` stands for: one
            // wait, half of the lanes at each barrier (a wait takes 100 cycles when nothing is left to wait for)
            auto wait_keys = [&](int j, uint64_t* bar, uint32_t parity) {
                const int st = halves ? j >> 1 : j, k = it + tc_pos_k(st, halves), b = k % kOps;
                const bool keys = j < items && (!halves || (j & 1) == 0) && (!bar || (lane & 1));
                return (!keys && !bar) || wait_all(keys ? &op_ready[b] : bar, keys ? uint32_t(k / kOps) & 1u : parity);
            };
            auto scores = [&](int j) {
                const int st = halves ? j >> 1 : j, t = j & 1, k = it + tc_pos_k(st, halves), b = k % kOps;
                tc_fence_after();
                const uint64_t ad = q_d + (halves && t ? C::kTile >> 4 : 0), bd = k_d + uint64_t(b * (C::kTile >> 4));
                if (elect_one()) {
                    umma_f16(tm + kColS + 128 * t, ad, bd, idesc_s, false);
#pragma unroll
                    for (int x = 1; x < D / 16; ++x) {
                        const uint32_t off = ((x >> 2) * C::kPlane + 32 * (x & 3)) >> 4;
                        umma_f16(tm + kColS + 128 * t, ad + off, bd + off, idesc_s, true);
                    }
                    umma_commit(&s_ready[t]);
                    if (!halves || t == 1) umma_commit(&op_free[b]);  // the tile's last use
                }
                __syncwarp();
            };
            for (int j = 0; ok && j < min(2, items); ++j) {
                ok = wait_keys(j, nullptr, 0);
                if (ok) scores(j);
            }
            for (int j = 0; ok && j < items; ++j) {
                const int st = halves ? j >> 1 : j, t = j & 1, k = it + tc_pos_v(st, n, halves), b = k % kOps;
                const uint64_t bd = v_d + uint64_t(b * (C::kTile >> 4));
                const uint32_t pp = t ? pph[1] : pph[0];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // before the first half the values, before the second the keys of the scores behind
                    const bool values = (!halves || t == 0) && (lane & 1);
                    ok = h == 0 ? wait_all(values ? &op_ready[b] : &p_ready[t][0], values ? uint32_t(k / kOps) & 1u : pp)
                                : wait_keys(j + 2, &p_ready[t][1], pp);
                    if (!ok) break;
                    __syncwarp();  // what one half of the lanes waited for, the issuing lane sees
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int x = 4 * h; x < 4 * h + 4; ++x)
                            umma_f16_ts(tm + kColO + 128 * t, tm + kColS + 128 * t + 8 * x, bd + ((2048 * x) >> 4),
                                        idesc_o, x > 0 || j > 1);
                        if (h == 1) {
                            if (!halves || t == 1) umma_commit(&op_free[b]);
                            if (j + 2 >= items) umma_commit(&o_done[t]);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (t)
                    pph[1] ^= 1u;
                else
                    pph[0] ^= 1u;
                if (j + 2 < items) scores(j + 2);
            }
            it += 2 * n;
        }
        // what was issued completes before tensor memory is freed, in a segment that was given up too
        __syncwarp();
        if (elect_one()) umma_commit(&mma_done);
        __syncwarp();
        (void)mbar_wait_bounded(&mma_done, 0, p.limit_ns);
    } else {
        // ---- softmax: tile t, thread = row = tensor memory lane
        const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lanes = uint32_t(wq * 32) << 16;
        const uint32_t tS = tmem + lanes + kColS + 128 * t, tO = tmem + lanes + kColO + 128 * t;
        const uint32_t flip = p.a.scale < 0.0f ? 0x80008000u : 0u;  // scores of -q, so that the scale is positive
        const float scale = fmaxf(fabsf(p.scale_log2), 1e-30f);     // not 0: -inf * 0 is no score
        uint32_t sph = 0, oph = 0;
        bool good = true;
        for (int sg = 0;; ++sg) {
            const int ss = sg % kTcSegs;
            bool ok = good && wait_all(&seg_full[ss], uint32_t(sg / kTcSegs) & 1u);
            const AttnSegment& g = seg_s[ss].g;
            const int n = ok ? (g.n + 1) / 2 : 0, rows = n ? min(kTcRows, g.T * p.group - g.row0) : 0;
            const bool halves = rows > 128;
            const int row = g.row0 + r + (halves ? 128 * t : 0);
            const bool mine = r + (halves ? 128 * t : 0) < rows;  // a row of the block
            const int ctx = g.ctx, len = ctx + g.T, end = (g.page0 + g.n) * kKvPage;
            uint64_t mask = 0;
            float m = kLowest, l = 0.0f;
            const int steps = n == 0 ? 0 : halves ? n : (n + 1 - t) / 2;  // of this tile
            if (n) {
                const int node = attn_row_token(p, row);
                if (mine) mask = p.a.mask ? __ldg(p.a.mask + g.t0 + node) : ~0ull >> (63 - node);
                if (halves || t == 0) {
                    const uint4* const src = reinterpret_cast<const uint4*>(
                        static_cast<const __half*>(p.a.q) + int64_t(g.t0 + node) * p.a.q_ld +
                        ((g.head - node) * p.group + row) * D);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        uint4 v = mine ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
                        v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
                        *reinterpret_cast<uint4*>(q_s + t * C::kTile + tc_chunk(r, c)) = v;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_ready[t]);
            }
            for (int i = 0; ok && i < steps; ++i) {
                ok = wait_all(&s_ready[t], sph);
                if (!ok) break;
                sph ^= 1u;
                tc_fence_after();
                const int key0 = g.page0 * kKvPage + (halves ? i : 2 * i + t) * kStep;
                // bit k of see[h]: the row sees key key0 + 64h + k
                uint64_t see[2];
                const bool tail = key0 + kStep > ctx || key0 + kStep > end;
                if (tail) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k0 = key0 + h * kKvPage, past = k0 - ctx;  // nodes before the page; < 0: context left
                        if (k0 >= min(end, len)) {
                            see[h] = 0;
                        } else if (past < 0) {
                            const uint64_t nodes = g.T < 64 ? mask & ((1ull << g.T) - 1) : mask;
                            see[h] = past <= -kKvPage ? ~0ull : ~0ull >> (kKvPage + past) | nodes << -past;
                        } else {  // past < 64, since k0 < len
                            see[h] = (g.T < 64 ? mask & ((1ull << g.T) - 1) : mask) >> past;
                        }
                    }
                }
                if (tail) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld32(tS + 32 * c, v);
                        tmem_ld_wait();
                        const uint32_t bits = uint32_t(see[c >> 1] >> (32 * (c & 1)));
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((bits >> k) & 1)) v[k] = 0xff800000u;
                        tmem_st32(tS + 32 * c, v);
                    }
                    tmem_st_wait();
                }
                // the maximum first, then the numbers again: tensor memory is read faster than registers spill
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[2][32];
                    tmem_ld32(tS + 64 * h, v[0]);
                    tmem_ld32(tS + 64 * h + 32, v[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        x0 = fmaxf(x0, __uint_as_float(v[0][k]));
                        x1 = fmaxf(x1, __uint_as_float(v[1][k]));
                    }
                }
                // raised for the lanes that need it; a row without keys so far keeps the lowest number
                const float top = fmaxf(x0, x1) * scale;
                const bool raise = top > m + kTcRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    const float mn = raise ? top : m, f = attn_factor(m - mn);
                    m = mn;
                    l *= f;
                    if (i > 0) {  // S is complete, so the product before it is: O is at rest
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st32(tO + 32 * c, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float base = kTcShift - m;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[2][32], pk[32];
                    tmem_ld32(tS + 64 * h, v[0]);
                    tmem_ld32(tS + 64 * h + 32, v[1]);
                    tmem_ld_wait();
                    float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float a = ex2(fmaf(__uint_as_float(v[k >> 4][2 * (k & 15)]), scale, base));
                        const float b = ex2(fmaf(__uint_as_float(v[k >> 4][2 * (k & 15) + 1]), scale, base));
                        l0 += a;
                        l1 += b;
                        pk[k] = pack_f16(a, b);
                    }
                    l += l0 + l1;
                    tmem_st32(tS + 32 * h, pk);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[t][h]);
                }
            }
            if (ok && steps > 0) {
                ok = wait_all(&o_done[t], oph);
                oph ^= 1u;
                tc_fence_after();
            }
            join_m[t][r] = m;
            join_l[t][r] = l;
            good = !barrier_any(1, 256, !ok);
            if (!good || n == 0) break;
            // ---- the outputs: of its own rows, or (steps in turn) tile 1's handed to tile 0
            const bool split = g.n_ctas > 1, both = !halves && n > 1;
            const bool odd = seg_s[ss].odd != 0, bad = seg_s[ss].bad != 0;
            float* const slot = p.parts + (int64_t(blockIdx.x) * 2 + g.slot) * attn_slot_floats(kTcRows, D);
            float f = 1.0f;
            if (both) {
                const float mo = join_m[t ^ 1][r], mm = fmaxf(m, mo);
                f = attn_factor(m - mm);
                l = l * f + join_l[t ^ 1][r] * attn_factor(mo - mm);
                m = mm;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const bool writes = mine && (halves || t == 0);
            const int at = row - g.row0;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                if (steps > 0) {
                    uint32_t v[32];
                    tmem_ld32(tO + 32 * c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(v[k]) * f;
                }
                if (both) {
                    if (t == 1) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) join[k * 128 + r] = o[k];
                    }
                    named_barrier_sync(1, 256);
                    if (t == 0) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] += join[k * 128 + r];
                    }
                    named_barrier_sync(1, 256);
                }
                if (writes && split) {
                    // [D/4][row][4], so that a warp's rows lie together
                    float4* const dst = reinterpret_cast<float4*>(slot + 2 * kTcRows) + (8 * c) * kTcRows + at;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[k * kTcRows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                } else if (writes && !bad) {
                    tc_emit(p, g, row, D, 32 * c, o, inv);
                }
                if (odd && writes && (split || !bad)) tc_add_dropped<D, Q8>(p, g, row, mask, 32 * c, split ? slot : nullptr);
            }
            if (writes && split) {
                slot[at] = m;
                slot[kTcRows + at] = bad ? kAttnBadPage : l;
            }
            if (!split && bad && threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
            tc_fence_before();  // the outputs are read: the next segment's products may follow the queries
            // the joining's plain writes come before the next queries', which the tensor cores read
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[ss]);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (abort_flag) {
        if (threadIdx.x == 0) atomicOr(status, MQ_DEV_TIMEOUT);
        float* const slots = p.parts + int64_t(blockIdx.x) * 2 * attn_slot_floats(kTcRows, D);
        if (threadIdx.x < kTcRows)
            slots[kTcRows + threadIdx.x] = slots[attn_slot_floats(kTcRows, D) + kTcRows + threadIdx.x] = kAttnGaveUp;
    }
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- the groups that several CTAs share: their parts joined in CTA order -------------------------
// CTA (first CTA of the group, 32 rows): a warp per 8 head values, a lane per row.  Bound by the parts' bytes, which
// lie in L2, where there are many rows, and by the latency of its loads where a group has many parts (38 of 14 rows
// for one sequence of 16000 tokens): so the values of four parts are on their way together, and before the maxima
// that they wait for; these go through shared memory, where all warps find them.  A kernel of its own, so that all
// SMs read them.
constexpr int kJoinAhead = 4;

template <int D>
__global__ void __launch_bounds__(4 * D, 1024 / (4 * D)) attn_tc_join_kernel(const AttnParams p, unsigned* status)
{
    extern __shared__ float part_s[];  // [parts][32] maxima, then sums
    __shared__ float top_s[D / 8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta0 = blockIdx.x;
    griddep_wait();
    const int4 s0 = __ldcg(p.shared + 2 * cta0), s1 = __ldcg(p.shared + 2 * cta0 + 1);
    const int n = s1.x, slab = blockIdx.y * 32, rows = min(kTcRows, s0.y * p.group - s0.w);
    if (n < 2 || slab >= rows) return;
    const bool mine = slab + lane < rows;
    const int row = min(slab + lane, rows - 1);
    const float* const first = p.parts + (int64_t(cta0) * 2 + s1.y) * attn_slot_floats(kTcRows, D);
    const float* const others = p.parts + int64_t(cta0) * 2 * attn_slot_floats(kTcRows, D);
    auto slot_of = [&](int c) { return c == 0 ? first : others + int64_t(c) * 2 * attn_slot_floats(kTcRows, D); };
    float4 x[kJoinAhead][2];
    auto load = [&](int c0) {
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const float4* const src =
                reinterpret_cast<const float4*>(slot_of(min(c0 + i, n - 1)) + 2 * kTcRows) + 2 * warp * kTcRows + row;
            x[i][0] = __ldcg(src);
            x[i][1] = __ldcg(src + kTcRows);
        }
    };
    load(0);
    float* const m_s = part_s;
    float* const l_s = part_s + n * 32;
    for (int c = warp; c < n; c += D / 8) {
        m_s[c * 32 + lane] = __ldcg(slot_of(c) + row);
        l_s[c * 32 + lane] = __ldcg(slot_of(c) + kTcRows + row);
    }
    __syncthreads();
    float mm = kLowest, l = 0.0f, o[8];
    bool gone = false, bad = false;
    for (int c = 0; c < n; ++c) mm = fmaxf(mm, m_s[c * 32 + lane]);
    for (int c = 0; c < n; ++c) {
        const float lc = l_s[c * 32 + lane];
        gone |= lc < 0.0f;
        bad |= lc == kAttnBadPage;
        l = fmaf(lc, attn_factor(m_s[c * 32 + lane] - mm), l);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.0f;
    for (int c0 = 0;;) {
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            if (c0 + i >= n) break;
            const float f = attn_factor(m_s[(c0 + i) * 32 + lane] - mm);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                o[4 * h] = fmaf(x[i][h].x, f, o[4 * h]);
                o[4 * h + 1] = fmaf(x[i][h].y, f, o[4 * h + 1]);
                o[4 * h + 2] = fmaf(x[i][h].z, f, o[4 * h + 2]);
                o[4 * h + 3] = fmaf(x[i][h].w, f, o[4 * h + 3]);
            }
        }
        c0 += kJoinAhead;
        if (c0 >= n) break;
        load(c0);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= inv;
    const int r = s0.w + row, node = attn_row_token(p, r), h = (s0.z - node) * p.group + r;
    const int64_t tok = s0.x + node;
    const int d0 = h * D + 8 * warp;
    const bool q8 = p.a.out_type != MQ_TYPE_F16;
    if (q8) {  // a block of 32 values lies in four warps
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(fabsf(o[i]))));
        top_s[warp][lane] = top;
        __syncthreads();
    }
    if (gone) {  // the group stays unwritten
        if (warp == 0 && bad) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    if (!mine) return;
    if (!q8) {
        *reinterpret_cast<uint4*>(static_cast<__half*>(p.a.out) + tok * p.a.out_ld + d0) =
            make_uint4(pack_f16(o[0], o[1]), pack_f16(o[2], o[3]), pack_f16(o[4], o[5]), pack_f16(o[6], o[7]));
        return;
    }
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(top_s[warp / 4 * 4 + i][lane]));
    const Q8Scale s = q8_scale_of(__uint_as_float(top));
    uint16_t* const dst = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.a.out) +
                                                      (tok * (p.a.n_heads * D / 32) + d0 / 32) * kQ8Bytes);
    if (warp % 4 == 0) dst[0] = __half_as_ushort(__float2half_rn(s.d));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int a, b;
        if (!q8_code_fast(o[2 * i], s, &a)) a = q8_code_exact(o[2 * i], s.d);
        if (!q8_code_fast(o[2 * i + 1], s, &b)) b = q8_code_exact(o[2 * i + 1], s.d);
        dst[1 + warp % 4 * 4 + i] = uint16_t((a & 255) | (b & 255) << 8);
    }
}

template <int D, bool Q8>
cudaError_t launch_tc(const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    attn_tc_kernel<D, Q8><<<grid, kTcThreads, TcCfg<D, Q8>::kSmem, s>>>(p, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;  // one CTA shares no group
    const int rows = p.group * p.a.max_tokens;
    return attn_launch_join(attn_tc_join_kernel<D>, dim3(grid, ((rows < kTcRows ? rows : kTcRows) + 31) / 32), 4 * D,
                            size_t(grid) * 2 * 32 * sizeof(float), p, status, s);  // 39 KB for 152 SMs
}

}  // namespace

int attn_tc_rows() { return kTcRows; }

cudaError_t launch_attn_tc(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    if (c.type == MQ_TYPE_Q8_0)
        return c.head_dim == 128 ? launch_tc<128, true>(p, grid, status, s)
                                 : launch_tc<64, true>(p, grid, status, s);
    return c.head_dim == 128 ? launch_tc<128, false>(p, grid, status, s)
                             : launch_tc<64, false>(p, grid, status, s);
}

cudaError_t set_attn_tc_attributes()
{
    cudaError_t e = cudaSuccess;
#define MQ_SET(D, Q)                                                                                              \
    if (e == cudaSuccess)                                                                                         \
        e = cudaFuncSetAttribute(attn_tc_kernel<D, Q>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<D, Q>::kSmem);
    MQ_SET(128, true) MQ_SET(64, true) MQ_SET(128, false) MQ_SET(64, false)
#undef MQ_SET
    return e;
}

}  // namespace mq
