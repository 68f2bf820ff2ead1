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
// turned by pos * inv_freq: a' = a cos - b sin, b' = b cos + a sin.  One warp
// per (token, run of heads): lane l holds elements 64j + 2l, +1, so loads and
// f16 stores are coalesced, a q8_0 block is half a warp's row, and the lane's
// cosines and sines (of the token alone) are formed once for all its heads.
// The partner of a pair comes through a row of shared memory, which serves
// every rot_dims and both pairings.  Statistics, products and rotation are
// fp32; each output is rounded once, to f16 or to its q8_0 code.
//
// The angle: pos * f / 2pi modulo one turn, with f = m 2^(e-23) (m the 24-bit
// mantissa): m * floor(2^64 / 2pi) is a 128-bit integer, shifted by e - 23 it
// is the turn per position as a 64-bit binary fraction, and the product with
// pos wraps exactly.  The fraction errs by about f units of 2^-64 per
// position, so the angle is good to fp32 at any position (pos * f rounded to
// fp32 is off by 4e-3 rad at position 131071).
__device__ __forceinline__ uint64_t turn_per_pos(float f)
{
    constexpr uint64_t kInv2Pi = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f);
    const int e = int((u >> 23) & 255u) - 127;
    uint64_t m = (u & 0x7fffffu) | 0x800000u;
    if (e < -100 || e > 63) return 0;  // zero, subnormal (no turn in 2^31 positions) or not a frequency
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

struct AppendArgs {
    mq_kv_append_args a;
    KvView c;
    int heads_per_warp, parts;  // runs of heads per token
};

template <int D, bool Q8>
__global__ void __launch_bounds__(128) kv_append_kernel(const AppendArgs p, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    constexpr int NJ = D / 64;  // element pairs per lane
    __shared__ float2 row_s[4][D / 2];
    const mq_kv_append_args& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t w = int64_t(blockIdx.x) * 4 + warp;
    const int n = int(w / p.parts), part = int(w - int64_t(n) * p.parts);
    if (n >= a.n_tokens) return;
    const int Hq = a.n_heads, Hkv = p.c.n_kv_heads, H = Hq + 2 * Hkv;
    const int h0 = part * p.heads_per_warp, h1 = min(h0 + p.heads_per_warp, H);

    // where K and V go: -1 writes q only
    int64_t page = -1;
    int r = 0;
    if (h1 > Hq) {
        const int slot = __ldg(a.slot + n);
        if (slot >= 0) {
            page = kv_page_of(p.c, __ldg(a.seq + n), slot, int64_t(Hkv) * B::kBytes);
            r = slot % kKvPage;
            if (page < 0 && lane == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        }
    }

    // cosine and signed sine of this lane's elements
    float cs[NJ][2], sn[NJ][2];
    int mate[NJ][2];
    const int R = a.rot_dims;
    const bool inter = (a.flags & MQ_ROPE_INTERLEAVED) != 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int d = 64 * j + 2 * lane + k;
            cs[j][k] = 1.0f, sn[j][k] = 0.0f, mate[j][k] = d;
            if (d < R && h0 < Hq + Hkv) {
                const int half = R / 2;
                const bool first = inter ? k == 0 : d < half;
                const int i = inter ? d / 2 : (first ? d : d - half);
                mate[j][k] = inter ? d ^ 1 : (first ? d + half : d - half);
                const uint64_t turn = turn_per_pos(__ldg(a.inv_freq + i)) * uint64_t(int64_t(__ldg(a.pos + n)));
                float s, c;
                sincospif(float(int(turn >> 32)) * 0x1p-31f, &s, &c);  // signed half turns
                cs[j][k] = c;
                sn[j][k] = first ? -s : s;
            }
        }

    const float2* const src = reinterpret_cast<const float2*>(a.qkv + size_t(n) * a.qkv_ld);
    float2 x[NJ], nx[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) nx[j] = __ldg(src + h0 * (D / 2) + 32 * j + lane);
    for (int h = h0; h < h1; ++h) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            x[j] = nx[j];
            if (h + 1 < h1) nx[j] = __ldg(src + (h + 1) * (D / 2) + 32 * j + lane);
        }
        const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
        if (!is_v) {
            const float* const wn = is_q ? a.q_norm : a.k_norm;
            if (wn) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) ss = fmaf(x[j].x, x[j].x, fmaf(x[j].y, x[j].y, ss));
#pragma unroll
                for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const float2 g = __ldg(reinterpret_cast<const float2*>(wn) + 32 * j + lane);
                    x[j].x = x[j].x * rs * g.x;
                    x[j].y = x[j].y * rs * g.y;
                }
            }
            if (R > 0) {
                float2* const row = row_s[warp];
#pragma unroll
                for (int j = 0; j < NJ; ++j) row[32 * j + lane] = x[j];
                __syncwarp();
                const float* const rowf = reinterpret_cast<const float*>(row);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    x[j].x = fmaf(x[j].x, cs[j][0], rowf[mate[j][0]] * sn[j][0]);
                    x[j].y = fmaf(x[j].y, cs[j][1], rowf[mate[j][1]] * sn[j][1]);
                }
                __syncwarp();
            }
        }
        if (is_q) {
            __half2* const q = reinterpret_cast<__half2*>(static_cast<__half*>(a.q_out) + size_t(n) * a.q_ld + h * D);
#pragma unroll
            for (int j = 0; j < NJ; ++j) q[32 * j + lane] = __floats2half2_rn(x[j].x, x[j].y);
            continue;
        }
        if (page < 0) continue;
        uint8_t* const blk = p.c.pages + page + size_t(is_v ? h - Hq - Hkv : h - Hq) * B::kBytes;
        uint8_t* const rows = blk + (is_v ? B::kVOff : 0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int d = 64 * j + 2 * lane;
            if (!Q8) {
                *reinterpret_cast<__half2*>(rows + B::chunk(r, d >> 3) + (d & 7) * 2) =
                    __floats2half2_rn(x[j].x, x[j].y);
                continue;
            }
            // a block of 32 values lies in 16 lanes; the bits of non-negative floats order like the values
            unsigned m = max(__float_as_uint(fabsf(x[j].x)), __float_as_uint(fabsf(x[j].y)));
#pragma unroll
            for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const Q8Scale s = q8_scale_of(__uint_as_float(m));
            int q0, q1;
            if (!q8_code_fast(x[j].x, s, &q0)) q0 = q8_code_exact(x[j].x, s.d);
            if (!q8_code_fast(x[j].y, s, &q1)) q1 = q8_code_exact(x[j].y, s.d);
            *reinterpret_cast<uchar2*>(rows + B::chunk(r, d >> 4) + (d & 15)) =
                make_uchar2(uint8_t(q0 + 128), uint8_t(q1 + 128));
            if ((lane & 15) == 0)
                *reinterpret_cast<__half*>(blk + B::kScK + (is_v ? B::kScBytes : 0) + (r * (D / 32) + (d >> 5)) * 2) =
                    __float2half_rn(s.d);
        }
    }
}

// ---- read ---------------------------------------------------------------------------------
// One thread per 16-byte chunk of a cached row: 16 bytes in, 16 (f16) or 32
// (q8_0, scale applied and rounded once) out, neighbouring threads on
// neighbouring chunks.  Bound by the bytes it moves.
template <int D, bool Q8>
__global__ void __launch_bounds__(256)
    kv_read_kernel(const KvView c, const int32_t* __restrict__ seq, const int32_t* __restrict__ slot, int n,
                   uint4* __restrict__ k_out, uint4* __restrict__ v_out, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    constexpr int CH = B::kChunks;
    const int64_t total = int64_t(n) * c.n_kv_heads * (2 * CH);
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += int64_t(gridDim.x) * blockDim.x) {
        const int ch = int(i % CH), is_v = int(i / CH) & 1;
        const int64_t th = i / (2 * CH);
        const int h = int(th % c.n_kv_heads), t = int(th / c.n_kv_heads);
        const int sl = __ldg(slot + t);
        const int64_t page = kv_page_of(c, __ldg(seq + t), sl, int64_t(c.n_kv_heads) * B::kBytes);
        if (page < 0) {
            atomicOr(status, MQ_DEV_KV_RANGE);
            continue;
        }
        const int r = sl % kKvPage;
        const uint8_t* const blk = c.pages + page + size_t(h) * B::kBytes;
        const uint4 v = *reinterpret_cast<const uint4*>(blk + (is_v ? B::kVOff : 0) + B::chunk(r, ch));
        uint4* const out = (is_v ? v_out : k_out) + th * (D / 8);
        if (!Q8) {
            out[ch] = v;
        } else {
            const uint32_t d = *reinterpret_cast<const uint16_t*>(blk + B::kScK + is_v * B::kScBytes +
                                                                  (r * (D / 32) + (ch >> 1)) * 2) * 0x10001u;
            uint32_t u[8];
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u[2 * k] = kv_pair(__byte_perm(in[k], 0x64646464u, 0x4140), d);
                u[2 * k + 1] = kv_pair(__byte_perm(in[k], 0x64646464u, 0x4342), d);
            }
            out[2 * ch] = make_uint4(u[0], u[1], u[2], u[3]);
            out[2 * ch + 1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
    }
}

// ---- accept -------------------------------------------------------------------------------
// One CTA per (sequence, head): every row of the path is read into registers
// before any is written, so the path may overlap its destination in any way.
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
    // one head per warp while that leaves the chip room (few tokens: latency), then
    // longer runs, which form a token's cosines and sines fewer times
    const int H = a.n_heads + 2 * cache.n_kv_heads;
    const int64_t per = int64_t(a.n_tokens) * H / (int64_t(num_sms) * 32);
    p.heads_per_warp = per < 1 ? 1 : per > 12 ? 12 : int(per);
    p.parts = (H + p.heads_per_warp - 1) / p.heads_per_warp;
    const int64_t grid = (int64_t(a.n_tokens) * p.parts + 3) / 4;
#define MQ_CALL(D, Q) kv_append_kernel<D, Q><<<unsigned(grid), 128, 0, s>>>(p, status)
    MQ_KV_DISPATCH(cache, MQ_CALL);
#undef MQ_CALL
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const mq_kv_cache& cache, const int32_t* seq, const int32_t* slot, int n, void* k_out,
                           void* v_out, int num_sms, unsigned* status, cudaStream_t s)
{
    const int ch = cache.head_dim / (cache.type == MQ_TYPE_Q8_0 ? 16 : 8);
    const int64_t total = int64_t(n) * cache.n_kv_heads * 2 * ch;
    int64_t grid = (total + 255) / 256;
    if (grid > int64_t(num_sms) * 64) grid = int64_t(num_sms) * 64;
#define MQ_CALL(D, Q)                                                                                              \
    kv_read_kernel<D, Q><<<unsigned(grid), 256, 0, s>>>(kv_view(cache), seq, slot, n, static_cast<uint4*>(k_out),  \
                                                        static_cast<uint4*>(v_out), status)
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
