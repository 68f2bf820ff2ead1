// attn_tc.cu -- attention of many query rows per key/value head (trees of more
// than a few tokens) over the paged cache, on the tensor cores.
//
// The same sums as attn.cu; with dozens to hundreds of query rows per
// key/value head every cached byte is used that often, and the products and
// the exponentials bound it instead of the cache's bytes.  Per CTA (one per
// SM, an equal share of all pages, mq_attn.cuh):
//   warps 0-3, 4-7  softmax of two tiles of 128 query rows, a thread per row
//   warps 8-11      q8_0: codes to f16 in the tensor cores' layout; both
//                   types: the values of pages that reach past the context
//                   made finite
//   warp 12         bulk copies of (page, head) blocks into a ring
//   warp 13         tensor memory; one lane issues the MMAs
// Tensor memory holds for each tile the queries (f16, the A operand), the
// scores of one page (64 columns), in their place the probabilities (f16, the
// A operand of the second product), and the fp32 outputs:
//   S[128][64] = Q K^T        K from shared memory, K-major
//   O[128][D] += P V          V from shared memory as it lies, MN-major
// so that shared memory is read for one operand only.  While one tile's
// probabilities are formed the other tile's products run: the issue order is
// S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...  With more than 128 rows the
// tiles are the rows' halves and both take every page; with fewer both hold
// the same rows, take the pages in turn and are joined at the end.
// Probabilities are 2^(s - m + 7) in f16, m the row's running maximum, which is
// raised (and O rescaled in tensor memory) only when a score passes it by more
// than 8, so they stay below 2^15; a key at 2^-21 of the largest is still a
// normal number.  Scores, maxima, sums and outputs are fp32.
#include "mq_attn.cuh"
#include "mq_umma.cuh"

namespace mq {

namespace {

constexpr int kTcRows = 256;  // query rows of a block
constexpr int kTcSegs = 4;
constexpr int kTcMaxStages = 12;
constexpr int kTcThreads = 448;
constexpr int kTcSmem = 218 * 1024;
constexpr float kTcRaise = 8.0f, kTcShift = 7.0f, kLowest = -3.402823466e38f;
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 384;  // tensor memory columns of tile 0; of tile 1 behind

template <int D, bool Q8>
struct TcCfg {
    using Raw = KvBlock<D, Q8>;
    using Op = KvBlock<D, false>;  // the operands' layout: an f16 block
    static constexpr int kJoin = 32 * 128 * 4;                // 32 outputs of 128 rows
    // q8_0: a ring of blocks as they come, and buffers of operands; f16: the ring's blocks are the operands
    static constexpr int kBufs = Q8 ? 3 : (kTcSmem - 1024 - kJoin) / Op::kBytes;
    static constexpr int kFit = (kTcSmem - 1024 - kJoin - kBufs * Op::kBytes) / Raw::kBytes;
    static constexpr int kStages = !Q8 ? kBufs : kFit < kTcMaxStages ? kFit : kTcMaxStages;
    static constexpr int kSmem = 1024 + kBufs * Op::kBytes + (Q8 ? kStages * Raw::kBytes : 0) + kJoin;
    static_assert(kStages >= 3 && kBufs <= 16 && kStages <= 16, "ring");
};

struct TcSegment {
    AttnSegment g;
    int odd, bad;  // a value that is not finite was dropped; a page outside the cache
};

// what a ring stage holds
struct TcPage {
    int key0, ctx, len, seg;
    int bad;
};

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

// ---- the values of one page, made operands (warps 8-11, thread x of 128) -----------------------
template <int D, bool Q8>
__device__ __forceinline__ bool tc_convert(const uint8_t* raw, uint8_t* op, const TcPage& pg, int x)
{
    using R = KvBlock<D, Q8>;
    using O = KvBlock<D, false>;
    const bool tail = pg.key0 + kKvPage > pg.ctx;
    bool odd = false;
    if (Q8) {
        constexpr int CH = D / 16;  // 16-code chunks of a row
        constexpr int kBatch = 4;   // loads in flight before the first store (which might be to the same place, for all
                                    // that the compiler knows)
#pragma unroll 1
        for (int i0 = 0; i0 < 2 * kKvPage * CH / 128; i0 += kBatch) {
            uint4 in[kBatch];
            uint32_t d[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int item = (i0 + i) * 128 + x, is_v = item / (kKvPage * CH), r = item / CH % kKvPage, c = item % CH;
                in[i] = lds16(raw + (is_v ? R::kVOff : 0) + R::chunk(r, c));
                d[i] = *reinterpret_cast<const uint16_t*>(raw + R::kScK + (is_v ? R::kScBytes : 0) +
                                                          (r * (D / 32) + (c >> 1)) * 2) * 0x10001u;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int item = (i0 + i) * 128 + x, is_v = item / (kKvPage * CH), r = item / CH % kKvPage, c = item % CH;
                const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
                uint32_t u[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    u[2 * k] = kv_pair(__byte_perm(w[k], 0x64646464u, 0x4140), d[i]);
                    u[2 * k + 1] = kv_pair(__byte_perm(w[k], 0x64646464u, 0x4342), d[i]);
                }
                if (tail && is_v) {
                    const bool out = pg.key0 + r >= pg.len;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (out) u[k] = 0;
                        if (pair_not_finite(u[k])) odd = true, u[k] = drop_pair(u[k]);
                    }
                }
                uint8_t* const dst = op + (is_v ? O::kVOff : 0);
                // the lanes of the second plane store their halves in the other order: no bank twice
                const bool swap = (c & 4) != 0;
                const uint4 lo = make_uint4(u[0], u[1], u[2], u[3]), hi = make_uint4(u[4], u[5], u[6], u[7]);
                *reinterpret_cast<uint4*>(dst + O::chunk(r, 2 * c + (swap ? 1 : 0))) = swap ? hi : lo;
                *reinterpret_cast<uint4*>(dst + O::chunk(r, 2 * c + (swap ? 0 : 1))) = swap ? lo : hi;
            }
        }
    } else if (tail) {
        for (int item = x; item < kKvPage * (D / 8); item += 128) {
            const int r = item / (D / 8);
            uint4* const v = reinterpret_cast<uint4*>(op + O::kVOff + O::chunk(r, item % (D / 8)));
            if (pg.key0 + r >= pg.len) {
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
    }
    return odd;
}

// the row's share of values that were dropped: what is not finite and seen makes the output what it is
template <int D, bool Q8>
__device__ __noinline__ void tc_add_dropped(const AttnParams& p, const AttnSegment& g, uint64_t mask, int d0,
                                            float (&o)[32])
{
    for (int pg = max(g.page0, g.ctx / kKvPage); pg < g.page0 + g.n; ++pg) {
        const int64_t page = kv_page_of(p.c, g.seq, pg * kKvPage, int64_t(p.c.n_kv_heads) * KvBlock<D, Q8>::kBytes);
        if (page < 0) continue;
        const uint8_t* const blk = p.c.pages + page + int64_t(g.head) * KvBlock<D, Q8>::kBytes;
        for (int r = 0; r < kKvPage; ++r) {
            const int j = pg * kKvPage + r;
            if (j >= g.ctx + g.T || (j >= g.ctx && !((mask >> (j - g.ctx)) & 1))) continue;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float v = kv_value<D, Q8>(blk, r, d0 + i, 1);
                if (!(v - v == 0.0f)) o[i] += v;
            }
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
    using Raw = typename C::Raw;
    using Op = typename C::Op;
    constexpr int kBufs = C::kBufs, kStages = C::kStages;
    extern __shared__ uint8_t sm_raw[];
    __shared__ __align__(8) uint64_t raw_full[kStages], raw_free[kStages], kv_ready[kBufs], kv_free[kBufs];
    __shared__ __align__(8) uint64_t q_ready[2], s_ready[2], p_ready[2], o_done[2], seg_full[kTcSegs], seg_empty[kTcSegs];
    __shared__ TcSegment seg_s[kTcSegs];
    __shared__ TcPage page_s[kStages];
    __shared__ float join_m[2][128], join_l[2][128];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the swizzled tiles want 1024-byte alignment
    uint8_t* const sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    uint8_t* const ops = sm;                                          // operand buffers (f16: the ring)
    uint8_t* const ring = Q8 ? sm + kBufs * Op::kBytes : sm;
    float* const join = reinterpret_cast<float*>(sm + kBufs * Op::kBytes + (Q8 ? kStages * Raw::kBytes : 0));

    if (threadIdx.x < kStages) {
        mbar_init(&raw_full[threadIdx.x], 1);
        mbar_init(&raw_free[threadIdx.x], 4);
    } else if (threadIdx.x >= 32 && threadIdx.x < 32 + kBufs) {
        mbar_init(&kv_ready[threadIdx.x - 32], 4);
        mbar_init(&kv_free[threadIdx.x - 32], 1);
    } else if (threadIdx.x >= 64 && threadIdx.x < 66) {
        const int k = threadIdx.x - 64;
        mbar_init(&q_ready[k], 4);
        mbar_init(&s_ready[k], 1);
        mbar_init(&p_ready[k], 4);
        mbar_init(&o_done[k], 1);
    } else if (threadIdx.x >= 96 && threadIdx.x < 96 + kTcSegs) {
        mbar_init(&seg_full[threadIdx.x - 96], 1);
        mbar_init(&seg_empty[threadIdx.x - 96], 8 + 4 + 1);  // softmax and converter warps, the MMA warp
        if (threadIdx.x == 96) abort_flag = 0;
    }
    fence_barrier_init();
    griddep_launch_dependents();  // the join may take its place; it waits for this grid's end
    AttnRange w;
    if (warp == 12) w = attn_range(p, kTcRows, status);
    if (warp == 13) tmem_alloc(&tmem_base, 512);
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

    if (warp == 12) {
        // ---- producer
        AttnSegment g = {};
        int at = w.first, it = 0, sg = 0, s = 0;
        uint32_t phase = 0;
        bool ok = true, more = true;
        for (; ok && more; ++sg) {
            more = attn_next(p, kTcRows, &w, &at, &g);
            if (!more) g.n = g.T = 0;
            const int ss = sg % kTcSegs;
            const int32_t* const table = p.c.table + int64_t(g.seq) * p.c.table_ld + g.page0;
            int32_t page_l = lane < g.n ? __ldg(table + lane) : 0;
            if (sg >= kTcSegs) ok = wait_all(&seg_empty[ss], uint32_t(sg / kTcSegs - 1) & 1u);
            if (!ok) break;
            if (lane == 0) {
                seg_s[ss].g = g;
                seg_s[ss].odd = seg_s[ss].bad = 0;
                mbar_arrive(&seg_full[ss]);
            }
            __syncwarp();
            for (int i0 = 0; ok && i0 < g.n; i0 += 32) {
                const int32_t page_now = page_l;
                if (i0 + 32 + lane < g.n) page_l = __ldg(table + i0 + 32 + lane);
                const int m = min(32, g.n - i0);
                for (int i = 0; i < m; ++i, ++it) {
                    const int32_t page = __shfl_sync(0xffffffffu, page_now, i);
                    // f16: the block is the operand, and the MMAs free it
                    if (it >= kStages) ok = wait_all(Q8 ? &raw_free[s] : &kv_free[s], phase ^ 1u);
                    if (!ok) break;
                    if (lane == 0) {
                        const bool bad = page < 0 || page >= p.c.n_pages;  // table entries are not trusted
                        page_s[s] = TcPage{(g.page0 + i0 + i) * kKvPage, g.ctx, g.ctx + g.T, ss, bad};
                        if (bad) {
                            mbar_arrive(&raw_full[s]);
                        } else {
                            mbar_arrive_expect_tx(&raw_full[s], Raw::kBytes);
                            bulk_copy_g2s(ring + s * Raw::kBytes,
                                          p.c.pages + (int64_t(page) * p.c.n_kv_heads + g.head) * Raw::kBytes,
                                          Raw::kBytes, &raw_full[s]);
                        }
                    }
                    if (++s == kStages) s = 0, phase ^= 1u;
                }
            }
        }
        // copies still in flight land before the CTA can exit
        for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
            (void)mbar_wait_bounded(&raw_full[j % kStages], uint32_t(j / kStages) & 1u, p.limit_ns);
    } else if (warp >= 8 && warp < 12) {
        // ---- operands: the pages in order, every segment's
        int s = 0, b = 0, it = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        for (int sg = 0; ok; ++sg) {
            const int ss = sg % kTcSegs;
            ok = wait_all(&seg_full[ss], uint32_t(sg / kTcSegs) & 1u);
            if (!ok) break;
            const int n = seg_s[ss].g.n;
            if (n == 0) break;
            for (int i = 0; i < n; ++i, ++it) {
                ok = wait_all(&raw_full[s], phase);
                if (Q8 && it >= kBufs) ok = ok && wait_all(&kv_free[b], bphase ^ 1u);
                if (!ok) break;
                const TcPage pg = page_s[s];
                uint8_t* const op = ops + (Q8 ? b * Op::kBytes : s * Op::kBytes);
                bool odd = false;
                if (!pg.bad) odd = tc_convert<D, Q8>(ring + s * Raw::kBytes, op, pg, (warp - 8) * 32 + lane);
                if (odd) seg_s[ss].odd = 1;
                if (pg.bad && lane == 0) seg_s[ss].bad = 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (Q8) mbar_arrive(&raw_free[s]);
                    mbar_arrive(&kv_ready[Q8 ? b : s]);
                }
                if (++s == kStages) s = 0, phase ^= 1u;
                if (++b == kBufs) b = 0, bphase ^= 1u;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[ss]);
        }
    } else if (warp == 13) {
        // ---- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc_s = umma_idesc_f16_f32(128, kKvPage);
            constexpr uint32_t idesc_o = umma_idesc_f16_f32(128, D) | kBMajorMn;
            // operand buffer 0; an address within it or in another is added to the descriptor's address field
            const uint64_t ops_k = umma_desc_sw128(smem_u32(ops)), ops_v = umma_desc_mn(smem_u32(ops) + Op::kVOff, kKvPage * 128);
            auto wait_one = [&](uint64_t* bar, uint32_t parity) {
                if (!abort_flag && mbar_wait_bounded(bar, parity, p.limit_ns)) return true;
                abort_flag = 1;
                return false;
            };
            int it = 0;              // pages before this segment
            uint32_t pph[2] = {0, 0}, qph = 0;  // phases of p_ready and q_ready
            bool ok = true;
            for (int sg = 0; ok; ++sg) {
                const int ss = sg % kTcSegs;
                ok = wait_one(&seg_full[ss], uint32_t(sg / kTcSegs) & 1u);
                if (!ok) break;
                const int n = seg_s[ss].g.n;
                if (n == 0) break;
                const bool halves = seg_s[ss].g.T * p.group - seg_s[ss].g.row0 > 128;
                const int items = halves ? 2 * n : n;
                mbar_arrive(&seg_empty[ss]);
                ok = wait_one(&q_ready[0], qph) && wait_one(&q_ready[1], qph);
                qph ^= 1u;
                int ready = 0;  // pages of the segment known to be there
                auto scores = [&](int j) {
                    const int pg = halves ? j >> 1 : j, t = j & 1, k = it + pg, b = k % kBufs;
                    if (pg >= ready) {
                        if (!wait_one(&kv_ready[b], uint32_t(k / kBufs) & 1u)) return false;
                        ready = pg + 1;
                    }
                    tc_fence_after();
                    const uint64_t kd = ops_k + uint64_t(b * (Op::kBytes >> 4));
                    umma_f16_ts(tmem + kColS + 64 * t, tmem + kColQ + 64 * t, kd, idesc_s, false);
#pragma unroll
                    for (int x = 1; x < D / 16; ++x)
                        umma_f16_ts(tmem + kColS + 64 * t, tmem + kColQ + 64 * t + 8 * x,
                                    kd + (((x >> 2) * (kKvPage * 128) + 32 * (x & 3)) >> 4), idesc_s, true);
                    umma_commit(&s_ready[t]);
                    return true;
                };
                for (int j = 0; ok && j < min(2, items); ++j) ok = scores(j);
                for (int j = 0; ok && j < items; ++j) {
                    const int pg = halves ? j >> 1 : j, t = j & 1, b = (it + pg) % kBufs;
                    ok = wait_one(&p_ready[t], pph[t]);
                    if (!ok) break;
                    pph[t] ^= 1u;
                    tc_fence_after();
                    const uint64_t vd = ops_v + uint64_t(b * (Op::kBytes >> 4));
                    umma_f16_ts(tmem + kColO + 128 * t, tmem + kColS + 64 * t, vd, idesc_o, j > 1);
#pragma unroll
                    for (int x = 1; x < kKvPage / 16; ++x)
                        umma_f16_ts(tmem + kColO + 128 * t, tmem + kColS + 64 * t + 8 * x, vd + ((2048 * x) >> 4), idesc_o,
                                    true);
                    if (!halves || t == 1) umma_commit(&kv_free[b]);  // the page's last use
                    if (j + 2 < items)
                        ok = scores(j + 2);
                    else
                        umma_commit(&o_done[t]);
                }
                it += n;
            }
            // what was issued completes before tensor memory is freed
            if (it > 0) (void)mbar_wait_bounded(&kv_free[(it - 1) % kBufs], uint32_t((it - 1) / kBufs) & 1u, p.limit_ns);
        }
    } else {
        // ---- softmax: tile t, thread = row = tensor memory lane
        const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lanes = uint32_t(wq * 32) << 16;
        const uint32_t tS = tmem + lanes + kColS + 64 * t, tO = tmem + lanes + kColO + 128 * t,
                       tQ = tmem + lanes + kColQ + 64 * t;
        const uint32_t flip = p.a.scale < 0.0f ? 0x80008000u : 0u;  // scores of -q, so that the scale is positive
        const float scale = fmaxf(fabsf(p.scale_log2), 1e-30f);     // not 0: -inf * 0 is no score
        uint32_t sph = 0, oph = 0;
        bool good = true;
        for (int sg = 0;; ++sg) {
            const int ss = sg % kTcSegs;
            bool ok = good && wait_all(&seg_full[ss], uint32_t(sg / kTcSegs) & 1u);
            const AttnSegment& g = seg_s[ss].g;
            const int n = ok ? g.n : 0, rows = n ? min(kTcRows, g.T * p.group - g.row0) : 0;
            const bool halves = rows > 128;
            const int row = g.row0 + r + (halves ? 128 * t : 0);
            const bool mine = r + (halves ? 128 * t : 0) < rows;  // a row of the block
            const int ctx = g.ctx, len = ctx + g.T;
            uint64_t mask = 0;
            float m = kLowest, l = 0.0f;
            const int steps = n == 0 ? 0 : halves ? n : (n + 1 - t) / 2;  // pages of this tile
            if (n) {
                const int node = attn_row_token(p, row);
                if (mine) mask = p.a.mask ? __ldg(p.a.mask + g.t0 + node) : ~0ull >> (63 - node);
                const uint4* const src = reinterpret_cast<const uint4*>(
                    static_cast<const __half*>(p.a.q) + int64_t(g.t0 + node) * p.a.q_ld +
                    ((g.head - node) * p.group + row) * D);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = mine ? __ldg(src + 8 * c + i) : make_uint4(0, 0, 0, 0);
                        v[4 * i] = x.x ^ flip, v[4 * i + 1] = x.y ^ flip, v[4 * i + 2] = x.z ^ flip, v[4 * i + 3] = x.w ^ flip;
                    }
                    tmem_st32(tQ + 32 * c, v);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_ready[t]);
            }
            for (int i = 0; ok && i < steps; ++i) {
                ok = wait_all(&s_ready[t], sph);
                if (!ok) break;
                sph ^= 1u;
                tc_fence_after();
                uint32_t v[2][32];
                tmem_ld32(tS, v[0]);
                tmem_ld32(tS + 32, v[1]);
                tmem_ld_wait();
                const int key0 = (g.page0 + (halves ? i : 2 * i + t)) * kKvPage;
                if (key0 + kKvPage > ctx) {
                    // bit k: the row sees key key0 + k
                    uint64_t see = key0 >= ctx ? 0 : ~0ull >> (kKvPage - (ctx - key0));  // ctx - key0 is 1..63
                    const int nodes = len - max(ctx, key0);  // tree nodes from the page's first on
                    uint64_t tree = key0 >= ctx ? (key0 - ctx < 64 ? mask >> (key0 - ctx) : 0) : mask << (ctx - key0);
                    if (nodes < 64) tree &= key0 >= ctx ? (1ull << nodes) - 1 : ((1ull << nodes) - 1) << (ctx - key0);
                    see |= tree;
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (!((see >> k) & 1)) v[k >> 5][k & 31] = 0xff800000u;
                }
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    x0 = fmaxf(x0, __uint_as_float(v[0][k]));
                    x1 = fmaxf(x1, __uint_as_float(v[1][k]));
                }
                // raised for the lanes that need it; a row without keys so far keeps the lowest number
                const float top = fmaxf(x0, x1) * scale;
                const bool raise = top > m + kTcRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    const float mn = raise ? top : m, f = ex2(m - mn);
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
                float l0 = 0.0f, l1 = 0.0f;
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float a = ex2(fmaf(__uint_as_float(v[k >> 4][2 * (k & 15)]), scale, base));
                    const float b = ex2(fmaf(__uint_as_float(v[k >> 4][2 * (k & 15) + 1]), scale, base));
                    l0 += a;
                    l1 += b;
                    pk[k] = pack_f16(a, b);
                }
                l += l0 + l1;
                tmem_st32(tS, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[t]);
            }
            if (ok && steps > 0) {
                ok = wait_all(&o_done[t], oph);
                oph ^= 1u;
                tc_fence_after();
            }
            join_m[t][r] = m;
            join_l[t][r] = l;
            good = !barrier_any(1, 256, !ok);
            if (!good) break;
            if (n == 0) break;
            // ---- the outputs: of its own rows, or (pages in turn) tile 1's handed to tile 0
            const bool split = g.n_ctas > 1;
            const bool odd = seg_s[ss].odd != 0, bad = seg_s[ss].bad != 0;
            float* const slot = p.parts + (int64_t(blockIdx.x) * 2 + g.slot) * attn_slot_floats(kTcRows, D);
            float f = 1.0f;
            if (!halves && n > 1) {
                const float mo = join_m[t ^ 1][r], mm = fmaxf(m, mo);
                f = ex2(m - mm);
                l = l * f + join_l[t ^ 1][r] * ex2(mo - mm);
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
                if (!halves && n > 1) {
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
                if (odd && writes) {
                    float add[32];  // a copy, so that the outputs stay in registers
#pragma unroll
                    for (int k = 0; k < 32; ++k) add[k] = 0.0f;
                    tc_add_dropped<D, Q8>(p, g, mask, 32 * c, add);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] += add[k];
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
            }
            if (writes && split) {
                slot[at] = m;
                slot[kTcRows + at] = bad ? -1.0f : l;
            }
            if (!split && bad && threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
            tc_fence_before();  // the outputs are read: the next segment's products may follow the queries
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[ss]);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (abort_flag && threadIdx.x == 0) atomicOr(status, MQ_DEV_TIMEOUT);
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- the groups that several CTAs share: their parts joined in CTA order -------------------------
// CTA (group, 32 rows), a warp per 32 head values, a thread per row of them.  Bound by the parts' bytes,
// which lie in L2; a kernel of its own, so that all SMs read them.
template <int D>
__global__ void __launch_bounds__(D) attn_tc_join_kernel(const AttnParams p, const int grid, unsigned* status)
{
    __shared__ AttnSegment g_s;
    __shared__ int there_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slab = blockIdx.x % (kTcRows / 32) * 32;
    if (warp == 0) {
        bool bad;
        const AttnRange w = attn_cut(p, kTcRows, grid, 0, &bad);
        AttnSegment g;
        const bool there = attn_group(p, kTcRows, w, blockIdx.x / (kTcRows / 32), &g);
        if (lane == 0) {
            there_s = there && g.n_ctas > 1;
            if (there_s) g_s = g;
        }
    }
    griddep_wait();
    __syncthreads();
    if (!there_s) return;
    const AttnSegment& g = g_s;
    const int row = slab + lane, rows = min(kTcRows, g.T * p.group - g.row0);
    if (row >= rows) return;
    auto slot_of = [&](int c) {
        return p.parts + (int64_t(g.cta0 + c) * 2 + (c == 0 ? g.slot0 : 0)) * attn_slot_floats(kTcRows, D);
    };
    float mm = kLowest, l = 0.0f, o[32];
    bool gone = false;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
#pragma unroll 8
    for (int c = 0; c < g.n_ctas; ++c) mm = fmaxf(mm, __ldcg(slot_of(c) + row));
#pragma unroll 2
    for (int c = 0; c < g.n_ctas; ++c) {
        const float* const slot = slot_of(c);
        const float lc = __ldcg(slot + kTcRows + row), f = ex2(__ldcg(slot + row) - mm);
        const float4* const src = reinterpret_cast<const float4*>(slot + 2 * kTcRows) + 8 * warp * kTcRows + row;
        gone |= lc < 0.0f;
        l = fmaf(lc, f, l);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 x = __ldcg(src + i * kTcRows);
            o[4 * i] = fmaf(x.x, f, o[4 * i]);
            o[4 * i + 1] = fmaf(x.y, f, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(x.z, f, o[4 * i + 2]);
            o[4 * i + 3] = fmaf(x.w, f, o[4 * i + 3]);
        }
    }
    if (gone) {  // a page outside the cache: the group stays unwritten
        atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    tc_emit(p, g, g.row0 + row, D, 32 * warp, o, l == 0.0f ? 0.0f : 1.0f / l);
}

template <int D, bool Q8>
cudaError_t launch_tc(const AttnParams& p, int grid, int64_t groups, unsigned* status, cudaStream_t s)
{
    attn_tc_kernel<D, Q8><<<grid, kTcThreads, TcCfg<D, Q8>::kSmem, s>>>(p, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;  // one CTA shares no group
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * (kTcRows / 32)));
    cfg.blockDim = dim3(D);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tc_join_kernel<D>, p, grid, status);
}

}  // namespace

int attn_tc_rows() { return kTcRows; }

cudaError_t launch_attn_tc(const mq_kv_cache& c, const AttnParams& p, int grid, unsigned* status, cudaStream_t s)
{
    const int64_t groups = int64_t(c.n_seqs) * c.n_kv_heads * ((p.group * p.a.max_tokens + kTcRows - 1) / kTcRows);
    if (c.type == MQ_TYPE_Q8_0)
        return c.head_dim == 128 ? launch_tc<128, true>(p, grid, groups, status, s)
                                 : launch_tc<64, true>(p, grid, groups, status, s);
    return c.head_dim == 128 ? launch_tc<128, false>(p, grid, groups, status, s)
                             : launch_tc<64, false>(p, grid, groups, status, s);
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
