// kv.cu -- the key/value cache: written with the per-head norms and the
// rotation in the same pass (kv_append), read back as f16 (kv_read), and a
// verified tree's accepted path moved to the end of the context (kv_accept).
#include <cuda_fp16.h>

#include "mq_internal.h"
#include "mq_kv.cuh"
#include "mq_stream.cuh"

namespace mq {

// ---- append -------------------------------------------------------------------------------
// Per head x[0..D): x' = x * rsqrt(mean(x^2) + eps) * w, then each pair (a, b)
// turned by pos * inv_freq: a' = a cos - b sin, b' = b cos + a sin.  Half a
// warp per head: lane l of 16 holds elements 4l..4l+3 (and 64 + 4l.. of 128),
// so loads and f16 stores are coalesced, a q8_0 block is eight lanes' share,
// and a pair lies in one lane (adjacent pairs; halves of 128), in lanes eight
// apart (halves of 64), or, where only part of the head turns by halves, comes
// through a row of shared memory.  A warp takes a run of pairs of heads of one
// token (query, key or value heads, so that its lanes agree on what to do) and
// forms the token's cosines and sines once.  Statistics, products and rotation
// are fp32; each output is rounded once, to f16 or to its q8_0 code.
//
// Measured (28 + 4 + 4 heads of 128, q8_0): one token 3.6 us, which is launch
// and one chain of loads, angles, norm and stores; 2048 tokens 16.0 us,
// 3.4 TB/s (f16 15.0): between instructions (the angles' sines, the q8_0 codes) and one
// wave's latency.
//
// The angle: pos * f / 2pi modulo one turn, with f = m 2^(e-23) (m the 24-bit
// mantissa): m * floor(2^64 / 2pi) is a 128-bit integer, shifted by e - 23 it
// is the turn per position as a 64-bit binary fraction, and the product with
// pos wraps exactly.  The fraction errs by at most f + 1 units of 2^-64 per
// position, so the angle is good to fp32 at any position for the frequencies
// of a rotation, 1 and below (pos * f rounded to fp32 is off by 4e-3 rad at
// position 131071).  From 2^64 on the product's low 64 bits say nothing: such
// a frequency, an infinity or NaN gives NaN (has_angle).
__device__ __forceinline__ uint64_t turn_per_pos(float f)
{
    constexpr uint64_t kInv2Pi = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f);
    const int e = int((u >> 23) & 255u) - 127;
    uint64_t m = (u & 0x7fffffu) | 0x800000u;
    if (e < -100 || e > 63) return 0;  // zero, subnormal (no turn in 2^31 positions); without an angle
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    const int sh = e - 23;  // left shift of hi:lo, modulo 2^64
    uint64_t t;
    if (sh >= 0)
        t = lo << sh;
    else if (sh > -64)
        t = (lo >> -sh) | (hi << (64 + sh));
    else
        t = sh > -128 ? hi >> (-sh - 64) : 0;
    return u >> 31 ? 0 - t : t;
}

__device__ __forceinline__ bool has_angle(float f) { return fabsf(f) < 0x1p64f; }

struct AppendArgs {
    mq_kv_append_args a;
    KvView c;
    int per_warp, parts;  // pairs of heads of a run, runs per token
    int wide;             // rows of qkv may be read 16 bytes at a time, rows of q written 8
};

enum { kRotNone = 0, kRotHalves = 1, kRotAdjacent = 2, kRotPart = 3 };

template <int D, bool Q8, int ROT>
__global__ void __launch_bounds__(128) kv_append_kernel(const AppendArgs p, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    constexpr int NV = D / 16, NG = NV / 4;  // values of a lane, groups of four
    __shared__ float row_s[ROT == kRotPart ? 8 : 1][D];
    const mq_kv_append_args& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15, hw = lane >> 4;
    const int64_t w = int64_t(blockIdx.x) * 4 + warp;
    const int n = int(w / p.parts), part = int(w - int64_t(n) * p.parts);
    if (n >= a.n_tokens) return;
    const int Hq = a.n_heads, Hkv = p.c.n_kv_heads;
    const int PQ = (Hq + 1) / 2, PK = (Hkv + 1) / 2;  // pairs
    const int p0 = part * p.per_warp, p1 = min(p0 + p.per_warp, PQ + 2 * PK);
    // pair i: 0 query, 1 key, 2 value heads; this half's head of that kind
    auto kind_of = [&](int i) { return i < PQ ? 0 : i < PQ + PK ? 1 : 2; };
    auto head_of = [&](int i, int kind) { return 2 * (i - (kind == 0 ? 0 : kind == 1 ? PQ : PQ + PK)) + hw; };

    const float* const src = a.qkv + size_t(n) * a.qkv_ld + 4 * l;
    auto load = [&](int i, float (&x)[NV]) {
        const int kind = kind_of(i), head = min(head_of(i, kind), (kind == 0 ? Hq : Hkv) - 1);
        const float* const from = src + (kind == 0 ? head : kind == 1 ? Hq + head : Hq + Hkv + head) * D;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const float* const at = from + 64 * j;
            if (p.wide) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(at));
                x[4 * j] = v.x, x[4 * j + 1] = v.y, x[4 * j + 2] = v.z, x[4 * j + 3] = v.w;
            } else {
                const float2 u = __ldg(reinterpret_cast<const float2*>(at)), v = __ldg(reinterpret_cast<const float2*>(at) + 1);
                x[4 * j] = u.x, x[4 * j + 1] = u.y, x[4 * j + 2] = v.x, x[4 * j + 3] = v.y;
            }
        }
    };
    float x[NV], nx[NV];
    load(p0, nx);

    // where K and V go: -1 writes q only
    int64_t page = -1;
    int r = 0;
    if (p1 > PQ) {
        const int slot = __ldg(a.slot + n);
        if (slot >= 0) {
            page = kv_page_of(p.c, __ldg(a.seq + n), slot, int64_t(Hkv) * B::kBytes);
            r = slot % kKvPage;
            if (page < 0 && lane == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        }
    }

    // cosine and signed sine of this lane's elements (halves of 128: of its first four, which its others share); what
    // lies beyond the rotated part is not multiplied by 1 and 0: an infinity would become NaN, and reach its neighbour
    constexpr int NC = ROT == kRotHalves && D == 128 ? 4 : NV;
    float cs[NC], sn[NC];
    int mate[ROT == kRotPart ? NV : 1];
    if (ROT != kRotNone && p0 < PQ + PK) {
        const int R = a.rot_dims, half = R / 2;
        const int64_t pos = __ldg(a.pos + n);
#pragma unroll
        for (int e = 0; e < NC; ++e) {
            const int d = 64 * (e / 4) + 4 * l + e % 4;
            cs[e] = 1.0f, sn[e] = 0.0f;
            if (ROT == kRotPart) mate[e] = d;
            // an adjacent pair shares its angle
            if (ROT == kRotAdjacent && (e & 1)) {
                cs[e] = cs[e - 1], sn[e] = -sn[e - 1];
                continue;
            }
            if (d < R) {
                const bool first = ROT == kRotAdjacent || d < half;
                const int i = ROT == kRotAdjacent ? d / 2 : (first ? d : d - half);
                if (ROT == kRotPart) mate[e] = first ? d + half : d - half;
                const float f = __ldg(a.inv_freq + i);
                const uint64_t turn = turn_per_pos(f) * uint64_t(pos);
                float s, c;
                sincospif(float(int(turn >> 32)) * 0x1p-31f, &s, &c);  // signed half turns
                if (!has_angle(f)) s = c = __uint_as_float(0x7fffffffu);
                cs[e] = c;
                sn[e] = first ? -s : s;
            }
        }
    }

    int wk = -1;  // kind whose weights are held
    float wt[NV];
#pragma unroll 1
    for (int i = p0; i < p1; ++i) {
        const int kind = kind_of(i), head = head_of(i, kind);
        const bool there = head < (kind == 0 ? Hq : Hkv);  // an odd number of heads leaves half a pair
#pragma unroll
        for (int e = 0; e < NV; ++e) x[e] = nx[e];
        if (i + 1 < p1) load(i + 1, nx);
        if (kind < 2) {
            const float* const wn = kind == 0 ? a.q_norm : a.k_norm;
            if (wn) {
                if (wk != kind) {
                    wk = kind;
#pragma unroll
                    for (int e = 0; e < NV; e += 2) {
                        const float2 g = __ldg(reinterpret_cast<const float2*>(wn + 64 * (e / 4) + 4 * l + e % 4));
                        wt[e] = g.x, wt[e + 1] = g.y;
                    }
                }
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < NV; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < NV; ++e) x[e] = x[e] * rs * wt[e];
            }
            if (ROT == kRotHalves && D == 128) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = x[e], v = x[e + NV - 4];  // sn[e] is the first of the pair's: -sin
                    x[e] = fmaf(u, cs[e], v * sn[e]);
                    x[e + NV - 4] = fmaf(v, cs[e], -(u * sn[e]));
                }
            } else if (ROT == kRotHalves) {
#pragma unroll
                for (int e = 0; e < NV; ++e) {
                    const float v = __shfl_xor_sync(0xffffffffu, x[e], 8);
                    x[e] = fmaf(x[e], cs[e % NC], v * sn[e % NC]);
                }
            } else if (ROT == kRotAdjacent) {
#pragma unroll
                for (int e = 0; e < NV; e += 2) {
                    if (64 * (e / 4) + 4 * l + e % 4 >= a.rot_dims) continue;
                    const float u = x[e], v = x[e + 1];
                    x[e] = fmaf(u, cs[e % NC], v * sn[e % NC]);
                    x[e + 1] = fmaf(v, cs[(e + 1) % NC], u * sn[(e + 1) % NC]);
                }
            } else if (ROT == kRotPart) {
                float* const row = row_s[2 * warp + hw];
#pragma unroll
                for (int e = 0; e < NV; ++e) row[64 * (e / 4) + 4 * l + e % 4] = x[e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < NV; ++e) {
                    const int d = 64 * (e / 4) + 4 * l + e % 4;
                    if (d < a.rot_dims) x[e] = fmaf(x[e], cs[e % NC], row[mate[e]] * sn[e % NC]);
                }
                __syncwarp();
            }
        }
        if (kind == 0) {
            if (!there) continue;
            __half* const q = static_cast<__half*>(a.q_out) + size_t(n) * a.q_ld + head * D + 4 * l;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const __half2 u = __floats2half2_rn(x[4 * j], x[4 * j + 1]), v = __floats2half2_rn(x[4 * j + 2], x[4 * j + 3]);
                __half2* const at = reinterpret_cast<__half2*>(q + 64 * j);
                if (p.wide) {
                    *reinterpret_cast<uint2*>(at) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
                } else {
                    at[0] = u, at[1] = v;
                }
            }
            continue;
        }
        if (page < 0) continue;
        uint8_t* const blk = p.c.pages + page + size_t(there ? head : 0) * B::kBytes;
        uint8_t* const rows = blk + (kind == 2 ? B::kVOff : 0);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int d = 64 * j + 4 * l;
            if (!Q8) {
                const __half2 u = __floats2half2_rn(x[4 * j], x[4 * j + 1]), v = __floats2half2_rn(x[4 * j + 2], x[4 * j + 3]);
                if (there)
                    *reinterpret_cast<uint2*>(rows + B::chunk(r, d >> 3) + (d & 7) * 2) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
                continue;
            }
            // a block of 32 values lies in eight lanes; the bits of non-negative floats order like the values
            unsigned m = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(fabsf(x[4 * j + e])));
#pragma unroll
            for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const Q8Scale s = q8_scale_of(__uint_as_float(m));
            uint32_t code = 0;
            bool sure = true;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                int q;
                sure &= q8_code_fast(x[4 * j + e], s, &q);
                code |= uint32_t(q + 128) << (8 * e);
            }
            if (!sure) {
                code = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) code |= uint32_t(q8_code_exact(x[4 * j + e], s.d) + 128) << (8 * e);
            }
            if (there) {
                *reinterpret_cast<uint32_t*>(rows + B::chunk(r, d >> 4) + (d & 15)) = code;
                if ((l & 7) == 0)
                    *reinterpret_cast<__half*>(blk + B::kScK + (kind == 2 ? B::kScBytes : 0) +
                                               (r * (D / 32) + (d >> 5)) * 2) = __float2half_rn(s.d);
            }
        }
    }
}

// ---- read ---------------------------------------------------------------------------------
// A thread per U 16-byte chunks of cached rows: 16 bytes in, 16 (f16) or 32
// (q8_0, scale applied and rounded once) out, neighbouring threads on
// neighbouring chunks of a token's heads.  Bound by the bytes it moves once
// enough of them are under way, by latency for few tokens.
struct ReadArgs {
    KvView c;
    const int32_t *seq, *slot;
    uint4 *k_out, *v_out;
    int n, per, tokens;  // pairs; chunks of a token, tokens of a CTA
    uint32_t per_inv;    // 2^32 / per rounded up
};
template <int D, bool Q8, int U>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadArgs p, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    constexpr int CH = B::kChunks;
    const int base = blockIdx.y * (256 * U) + threadIdx.x;
    uint4 v[U];
    uint32_t d[U];
    uint4* out[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        out[i] = nullptr;
        const int x = base + 256 * i;
        // x / per, exact: x < 2^16 where a CTA has several tokens, and one token is all of x otherwise
        const int tl = p.tokens > 1 ? int(__umulhi(uint32_t(x), p.per_inv)) : 0, u = x - tl * p.per;
        const int64_t t = int64_t(blockIdx.x) * p.tokens + tl;
        if (tl >= p.tokens || u >= p.per || t >= p.n) continue;
        const int sl = __ldg(p.slot + t), r = sl & (kKvPage - 1);
        const int64_t page = kv_page_of(p.c, __ldg(p.seq + t), sl, int64_t(p.c.n_kv_heads) * B::kBytes);
        if (page < 0) {
            if (u == 0) atomicOr(status, MQ_DEV_KV_RANGE);
            continue;
        }
        const int ch = u % CH, is_v = u / CH & 1, h = u / (2 * CH);
        const uint8_t* const blk = p.c.pages + page + size_t(h) * B::kBytes;
        v[i] = *reinterpret_cast<const uint4*>(blk + (is_v ? B::kVOff : 0) + B::chunk(r, ch));
        if (Q8)
            d[i] = *reinterpret_cast<const uint16_t*>(blk + B::kScK + is_v * B::kScBytes +
                                                      (r * (D / 32) + (ch >> 1)) * 2) * 0x10001u;
        out[i] = (is_v ? p.v_out : p.k_out) + (t * p.c.n_kv_heads + h) * (D / 8) + (Q8 ? 2 * ch : ch);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (!out[i]) continue;
        if (!Q8) {
            *out[i] = v[i];
            continue;
        }
        uint32_t o[8];
        const uint32_t in[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[2 * k] = kv_pair(__byte_perm(in[k], 0x64646464u, 0x4140), d[i]);
            o[2 * k + 1] = kv_pair(__byte_perm(in[k], 0x64646464u, 0x4342), d[i]);
        }
        out[i][0] = make_uint4(o[0], o[1], o[2], o[3]);
        out[i][1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// ---- accept -------------------------------------------------------------------------------
// One CTA per (sequence, head): every row of the path is read into registers
// before any is written, so the path may overlap its destination in any way.
// Bound by latency: one sequence 2.7 us, 64 of them 3.2 us (11 nodes, f16).
template <int D, bool Q8>
__global__ void __launch_bounds__(256)
    kv_accept_kernel(const KvView c, const int32_t* __restrict__ ctx_len, const int32_t* __restrict__ path,
                     const int32_t* __restrict__ n_path, int path_ld, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    constexpr int CH = 2 * B::kChunks;                                // K's and V's chunks of a row
    constexpr int kPer = (MQ_TREE_MAX_TOKENS * CH + 255) / 256;       // chunks per thread
    constexpr int kSc = 2 * (D / 32);                                 // scales of a row
    constexpr int kScPer = (MQ_TREE_MAX_TOKENS * kSc + 255) / 256;
    __shared__ int64_t src_s[MQ_TREE_MAX_TOKENS], dst_s[MQ_TREE_MAX_TOKENS];  // block offset | row
    __shared__ uint8_t srow_s[MQ_TREE_MAX_TOKENS], drow_s[MQ_TREE_MAX_TOKENS];
    const int s = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int n = __ldg(n_path + s), ctx = __ldg(ctx_len + s);
    bool bad = n < 0 || n > path_ld || ctx < 0 || ctx > c.table_ld * int64_t(kKvPage) - n;
    if (!bad && tid < n) {
        const int64_t page_bytes = int64_t(c.n_kv_heads) * B::kBytes;
        const int node = __ldg(path + int64_t(s) * path_ld + tid);
        const int from = ctx + (node & (MQ_TREE_MAX_TOKENS - 1)), to = ctx + tid;
        bad = node < 0 || node >= MQ_TREE_MAX_TOKENS;
        const int64_t a = kv_page_of(c, s, from, page_bytes), b = kv_page_of(c, s, to, page_bytes);
        bad = bad || a < 0 || b < 0;
        src_s[tid] = a + int64_t(h) * B::kBytes;
        dst_s[tid] = b + int64_t(h) * B::kBytes;
        srow_s[tid] = uint8_t(from % kKvPage);
        drow_s[tid] = uint8_t(to % kKvPage);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    uint4 v[kPer];
    uint16_t sc[kScPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = k * 256 + tid, row = i / CH, ch = i % CH;
        if (row < n)
            v[k] = *reinterpret_cast<const uint4*>(c.pages + src_s[row] + (ch >= B::kChunks ? B::kVOff : 0) +
                                                   B::chunk(srow_s[row], ch % B::kChunks));
    }
    if (Q8) {
#pragma unroll
        for (int k = 0; k < kScPer; ++k) {
            const int i = k * 256 + tid, row = i / kSc, e = i % kSc;
            if (row < n)
                sc[k] = *reinterpret_cast<const uint16_t*>(c.pages + src_s[row] + B::kScK +
                                                           (e >= D / 32 ? B::kScBytes : 0) +
                                                           (srow_s[row] * (D / 32) + e % (D / 32)) * 2);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = k * 256 + tid, row = i / CH, ch = i % CH;
        if (row < n)
            *reinterpret_cast<uint4*>(c.pages + dst_s[row] + (ch >= B::kChunks ? B::kVOff : 0) +
                                      B::chunk(drow_s[row], ch % B::kChunks)) = v[k];
    }
    if (Q8) {
#pragma unroll
        for (int k = 0; k < kScPer; ++k) {
            const int i = k * 256 + tid, row = i / kSc, e = i % kSc;
            if (row < n)
                *reinterpret_cast<uint16_t*>(c.pages + dst_s[row] + B::kScK + (e >= D / 32 ? B::kScBytes : 0) +
                                             (drow_s[row] * (D / 32) + e % (D / 32)) * 2) = sc[k];
        }
    }
}

// ---- launchers ----------------------------------------------------------------------------
#define MQ_KV_DISPATCH(cache, CALL)                       \
    do {                                                  \
        if ((cache).type == MQ_TYPE_Q8_0) {               \
            if ((cache).head_dim == 128) { CALL(128, true); } else { CALL(64, true); }   \
        } else {                                          \
            if ((cache).head_dim == 128) { CALL(128, false); } else { CALL(64, false); } \
        }                                                 \
    } while (0)

cudaError_t launch_kv_append(const mq_kv_cache& cache, const mq_kv_append_args& a, int num_sms, unsigned* status,
                             cudaStream_t s)
{
    AppendArgs p;
    p.a = a;
    p.c = kv_view(cache);
    // a pair of heads per warp while that leaves the chip room (few tokens: latency), then longer runs, which
    // form a token's cosines and sines fewer times: 2048 tokens of 36 heads take 30, 22, 20, 16 and 21 us in
    // runs of one, two, four, nine and 18 pairs.  Measured with those 18 pairs alone, which nine halves; other
    // numbers of heads get the fewest runs of at most nine, of one length
    const int pairs = (a.n_heads + 1) / 2 + 2 * ((cache.n_kv_heads + 1) / 2);
    const int64_t per = int64_t(a.n_tokens) * pairs / (int64_t(num_sms) * 16);
    p.per_warp = per < 1 ? 1 : per > 9 ? 9 : int(per);
    p.parts = (pairs + p.per_warp - 1) / p.per_warp;
    p.per_warp = (pairs + p.parts - 1) / p.parts;  // runs of the same length, and none of length zero
    p.parts = (pairs + p.per_warp - 1) / p.per_warp;
    p.wide = (reinterpret_cast<uintptr_t>(a.qkv) & 15) == 0 && a.qkv_ld % 4 == 0 &&
             (reinterpret_cast<uintptr_t>(a.q_out) & 7) == 0 && a.q_ld % 4 == 0;
    const unsigned grid = unsigned((int64_t(a.n_tokens) * p.parts + 3) / 4);
    const int rot = a.rot_dims == 0 ? kRotNone : a.flags & MQ_ROPE_INTERLEAVED ? kRotAdjacent
                    : a.rot_dims == cache.head_dim ? kRotHalves : kRotPart;
#define MQ_CALL(D, Q)                                                                                           \
    rot == kRotNone ? kv_append_kernel<D, Q, kRotNone><<<grid, 128, 0, s>>>(p, status)                          \
    : rot == kRotHalves ? kv_append_kernel<D, Q, kRotHalves><<<grid, 128, 0, s>>>(p, status)                    \
    : rot == kRotAdjacent ? kv_append_kernel<D, Q, kRotAdjacent><<<grid, 128, 0, s>>>(p, status)                \
                          : kv_append_kernel<D, Q, kRotPart><<<grid, 128, 0, s>>>(p, status)
    MQ_KV_DISPATCH(cache, MQ_CALL);
#undef MQ_CALL
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const mq_kv_cache& cache, const int32_t* seq, const int32_t* slot, int n, void* k_out,
                           void* v_out, int num_sms, unsigned* status, cudaStream_t s)
{
    ReadArgs p;
    p.c = kv_view(cache);
    p.seq = seq, p.slot = slot;
    p.k_out = static_cast<uint4*>(k_out), p.v_out = static_cast<uint4*>(v_out);
    p.n = n;
    p.per = cache.n_kv_heads * 2 * (cache.head_dim / (cache.type == MQ_TYPE_Q8_0 ? 16 : 8));
    p.per_inv = uint32_t((0x100000000ull + p.per - 1) / p.per);
    // Four chunks per thread once the chip has plenty of them; with 4 heads of 128 and one or four: f16, 4096 tokens
    // 3.9 and 4.6 us, 16384 17.6 and 13.5, 131072 119 and 84 (6.4 TB/s); q8_0, 32768 22.3 (4.6 TB/s) and 24.1, 131072 79
    // and 76.  Other head counts and heads of 64 were not measured; the rule counts their chunks alike.
    const bool many = int64_t(n) * p.per >= int64_t(num_sms) * (cache.type == MQ_TYPE_Q8_0 ? 20480 : 8192);
    const int chunks = many ? 1024 : 256;  // of a CTA
    p.tokens = p.per < chunks ? chunks / p.per : 1;
    const dim3 grid(unsigned((int64_t(n) + p.tokens - 1) / p.tokens), unsigned((p.per + chunks - 1) / chunks));
#define MQ_CALL(D, Q)                                                           \
    many ? kv_read_kernel<D, Q, 4><<<grid, 256, 0, s>>>(p, status)              \
         : kv_read_kernel<D, Q, 1><<<grid, 256, 0, s>>>(p, status)
    MQ_KV_DISPATCH(cache, MQ_CALL);
#undef MQ_CALL
    return cudaGetLastError();
}

cudaError_t launch_kv_accept(const mq_kv_cache& cache, const int32_t* ctx_len, const int32_t* path,
                             const int32_t* n_path, int path_ld, unsigned* status, cudaStream_t s)
{
    const dim3 grid(unsigned(cache.n_seqs), unsigned(cache.n_kv_heads));
#define MQ_CALL(D, Q) \
    kv_accept_kernel<D, Q><<<grid, 256, 0, s>>>(kv_view(cache), ctx_len, path, n_path, path_ld, status)
    MQ_KV_DISPATCH(cache, MQ_CALL);
#undef MQ_CALL
    return cudaGetLastError();
}

}  // namespace mq
