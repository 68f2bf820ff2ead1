// attn.cu -- attention of drafted token trees over the paged cache.
//
// Per (token, head): s_j = scale * q.k_j over the keys the node sees,
// out = sum_j exp(s_j - max) v_j / sum_j exp(s_j - max), with the running
// maximum and sum of one pass over the cache.
//
// One CTA of four warps per (token, head): warp w takes keys w, w+4, ...,
// each lane holding D/32 of the head's values; the warps' partial maxima,
// sums and outputs are joined at the end.
#include <cuda_fp16.h>

#include "mq_internal.h"
#include "mq_kv.cuh"
#include "mq_stream.cuh"

namespace mq {

struct AttnParams {
    mq_attn_args a;
    KvView c;
    int group;  // query heads per key/value head
};

template <int D, bool Q8>
__device__ __forceinline__ float kv_value(const uint8_t* blk, int r, int d, int is_v)
{
    using B = KvBlock<D, Q8>;
    const uint8_t* const rows = blk + (is_v ? B::kVOff : 0);
    if (!Q8) return __half2float(*reinterpret_cast<const __half*>(rows + B::chunk(r, d >> 3) + (d & 7) * 2));
    const __half sc =
        *reinterpret_cast<const __half*>(blk + B::kScK + is_v * B::kScBytes + (r * (D / 32) + (d >> 5)) * 2);
    return __half2float(__hmul(__int2half_rn(int(rows[B::chunk(r, d >> 4) + (d & 15)]) - 128), sc));
}

template <int D, bool Q8>
__global__ void __launch_bounds__(128) attn_kernel(const AttnParams p, unsigned* status)
{
    using B = KvBlock<D, Q8>;
    constexpr int E = D / 32;
    __shared__ float m_s[4], l_s[4], o_s[4][D];
    const int n = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const mq_attn_args& a = p.a;
    // the token's sequence
    int seq = -1;
    for (int s = 0; s < p.c.n_seqs; ++s)
        if (n >= a.tok_start[s] && n < a.tok_start[s + 1]) seq = s;
    if (n == 0 && h == 0 && threadIdx.x == 0)
        for (int s = 0; s < p.c.n_seqs; ++s)
            if (a.tok_start[s + 1] < a.tok_start[s]) atomicOr(status, MQ_DEV_KV_RANGE);
    if (seq < 0) return;
    const int t0 = a.tok_start[seq], T = a.tok_start[seq + 1] - t0, ctx = a.ctx_len[seq], node = n - t0;
    if (t0 < 0 || T > a.max_tokens || ctx < 0 || int64_t(ctx) + T > a.max_len) {
        if (threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    const uint64_t mask = a.mask ? a.mask[n] : ~0ull >> (63 - node);
    float q[E], o[E];
    for (int e = 0; e < E; ++e) {
        q[e] = __half2float(static_cast<const __half*>(a.q)[size_t(n) * a.q_ld + h * D + lane + 32 * e]) * a.scale;
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    bool bad = false;
    for (int j = warp; j < ctx + T; j += 4) {
        if (j >= ctx && !((mask >> (j - ctx)) & 1)) continue;
        const int64_t page = kv_page_of(p.c, seq, j, int64_t(p.c.n_kv_heads) * B::kBytes);
        if (page < 0) {
            bad = true;
            break;
        }
        const uint8_t* const blk = p.c.pages + page + size_t(h / p.group) * B::kBytes;
        const int r = j % kKvPage;
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], kv_value<D, Q8>(blk, r, lane + 32 * e, 0), s);
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.0f : expf(m - mn), w = s == -INFINITY ? 0.0f : expf(s - mn);
        l = l * f + w;
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, kv_value<D, Q8>(blk, r, lane + 32 * e, 1), o[e] * f);
        m = mn;
    }
    if (lane == 0) m_s[warp] = m, l_s[warp] = l;
    for (int e = 0; e < E; ++e) o_s[warp][lane + 32 * e] = o[e];
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(status, MQ_DEV_KV_RANGE);
        return;
    }
    const int d = threadIdx.x;
    if (d >= D) return;
    float mm = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3])), sum = 0.0f, val = 0.0f;
    for (int w = 0; w < 4; ++w) {
        const float f = m_s[w] == -INFINITY ? 0.0f : expf(m_s[w] - mm);
        sum += l_s[w] * f;
        val += l_s[w] == 0.0f ? 0.0f : o_s[w][d] * f;
    }
    val = sum == 0.0f ? 0.0f : val / sum;
    if (a.out_type == MQ_TYPE_F16) {
        static_cast<__half*>(a.out)[size_t(n) * a.out_ld + h * D + d] = __float2half_rn(val);
    } else {
        float sc;
        const int code = q8_quantize_lane(val, &sc);
        uint8_t* const ob =
            static_cast<uint8_t*>(a.out) + (size_t(n) * (a.n_heads * D / 32) + h * (D / 32) + warp) * kQ8Bytes;
        if (lane == 0) *reinterpret_cast<__half*>(ob) = __float2half_rn(sc);
        ob[2 + lane] = uint8_t(int8_t(code));
    }
}

size_t attn_workspace_bytes(const mq_kv_cache&, int, int, int) { return 128; }

cudaError_t launch_attn(const mq_kv_cache& cache, const mq_attn_args& a, void*, int, unsigned* status, cudaStream_t s)
{
    const AttnParams p{a, kv_view(cache), a.n_heads / cache.n_kv_heads};
    const dim3 grid(unsigned(a.n_tokens), unsigned(a.n_heads));
    if (cache.type == MQ_TYPE_Q8_0) {
        if (cache.head_dim == 128)
            attn_kernel<128, true><<<grid, 128, 0, s>>>(p, status);
        else
            attn_kernel<64, true><<<grid, 128, 0, s>>>(p, status);
    } else {
        if (cache.head_dim == 128)
            attn_kernel<128, false><<<grid, 128, 0, s>>>(p, status);
        else
            attn_kernel<64, false><<<grid, 128, 0, s>>>(p, status);
    }
    return cudaGetLastError();
}

}  // namespace mq
