// softmax.cu -- y = softmax(scale * x) of fp32 rows: the target's probabilities
// from the logits of every node of a step.
//
//   y_i = 2^((x_i - m) k) / sum_j 2^((x_j - m) k),   m = max x,  k = scale * log2(e)
//
// Bound by its bytes, so a row passes through the chip once: a cluster of up to
// eight CTAs holds it in registers.  Each CTA forms its own maximum and, with
// that, its exponentials and their sum; the (maximum, sum) pairs go round the
// cluster through distributed shared memory (one barrier), and what is left is a
// factor per CTA.  Rows longer than eight CTAs hold (147456 values, 147450 where
// rows start anywhere) are read twice: from L2 while the rows on the chip at once,
// up to 76, fit into it, which ends at some 420000 values a row; from HBM beyond.
// A CTA calls for the part of a later row when it starts, so HBM is read while
// others reduce and store.  Measured: 512 x 131072 98 us, 5.5 TB/s; 512 x 131071
// 108, 512 x 50001 46, 7 x 50001 4.2.  An earlier form took 124 us for the first
// without the prefetch and 110 with it, and 244 with one CTA per SM.
// Clusters of 16, which would hold rows of up to 262144, are slower to place: 256 x
// 200003 140 us, read twice by clusters of eight 117; 512 x 131071 240.
// Maxima, exponentials and sums are fp32; x - m, its product with k and k itself
// are rounded once each, relative to |x - m|, and the exponential is the hardware's
// (2^-22).  Normal logits, 512 x 131072: the largest relative error of an output is
// 2.5e-6, where exp(x - m) by itself in fp32 has 1.2e-6.  With k in two parts it was
// 2.35e-6 and 104 us; with exp2f as well a value took 31 instructions, whose issue
// bound the kernel.
#include <cooperative_groups.h>

#include "mq_internal.h"
#include "mq_tma.cuh"

namespace mq {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCluster = 8;

struct SoftmaxArgs {
    const float* x;
    float* y;
    int64_t x_ld, y_ld;
    int vocab;
    float k;  // scale * log2(e), or twice that (H)
    int rows, ahead;  // rows that are on the chip at once: a later one's part is called for when a CTA starts
};

// 2^((x - m) k), mh = m, or with H of halves and mh = m / 2: -inf gives 0, NaN stays.  A difference that passes the
// largest number, 3.4e38, weighs something at scales below some 3e-37 only: H is for those (x - m is rounded once all
// the same).  For every scale it cost 512 x 131072 2 us of 98.
template <bool H>
__device__ __forceinline__ float exp_of(float x, float mh, const SoftmaxArgs& p)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((H ? fmaf(x, 0.5f, -mh) : x - mh) * p.k));
    return y;
}

// A larger maximum scales a sum by this; of a part that saw nothing (maximum -inf beside a finite one), 0.
template <bool H>
__device__ __forceinline__ float factor(float m, float top, const SoftmaxArgs& p)
{
    return m == top ? 1.0f : exp_of<H>(m, H ? top * 0.5f : top, p);
}

// maximum or sum over the CTA
template <bool Max>
__device__ __forceinline__ float cta_reduce(float v, float* s)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = Max ? fmaxf(v, w) : v + w;
    }
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) v = Max ? fmaxf(v, s[i]) : v + s[i];
    return v;
}

// NV > 0: the CTA's part of the row is up to 4 * NV values per thread, in registers; 0: any length, read twice
// Several CTAs per SM, so that some load while others reduce or store.
template <int NV, bool H>
__global__ void __launch_bounds__(kThreads, NV >= 4 ? 2 : 4) softmax_kernel(const SoftmaxArgs p)
{
    constexpr float h = H ? 0.5f : 1.0f;
    __shared__ float max_s[kWarps], sum_s[kWarps];
    __shared__ float2 part_s[kMaxCluster];  // every CTA's maximum and sum
    cg::cluster_group cl = cg::this_cluster();
    // the others' shared memory is written once they run; nothing else has to be seen, so no fence
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    const int64_t row = blockIdx.x / C;
    const float* const x = p.x + row * p.x_ld;
    float* const y = p.y + row * p.y_ld;
    // units of four values that start at 16-byte boundaries of x: unit u holds the values 4u - off .. 4u - off + 3
    const int off = int(reinterpret_cast<uintptr_t>(x) >> 2) & 3;
    const int units = int((int64_t(p.vocab) + off + 3) / 4), per = (units + C - 1) / C;
    const int first = rank * per, last = min(units, first + per);
    const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15) == 0;
    auto load = [&](int u, float (&v)[4]) {
        const int i = 4 * u - off;
        if (i >= 0 && i <= p.vocab - 4) {
            const float4 w = __ldcs(reinterpret_cast<const float4*>(x + i));
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = i + e >= 0 && i + e < p.vocab ? x[i + e] : -INFINITY;
        }
    };
    auto store = [&](int u, const float (&v)[4]) {
        const int i = 4 * u - off;
        if (same && i >= 0 && i <= p.vocab - 4) {
            *reinterpret_cast<float4*>(y + i) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e >= 0 && i + e < p.vocab) y[i + e] = v[e];
        }
    };
    if (threadIdx.x == 0 && row + p.ahead < p.rows && NV >= 4) {
        const float* const next = x + p.ahead * p.x_ld;
        const int o = int(reinterpret_cast<uintptr_t>(next) >> 2) & 3, from = 4 * first > o ? 4 * first : 4;
        const int to = min(4 * last, p.vocab + o) & ~3;
        if (from < to) prefetch_l2(next + (from - o), uint32_t(to - from) * 4);
    }
    float v[NV > 0 ? NV : 1][4];
    float m = -INFINITY, l = 0.0f;
    // no unit of the part reaches past the row's ends: no test per unit but that there is one
    const bool inner = same && 4 * first >= off && 4 * last - off <= p.vocab;
    if constexpr (NV > 0) {
        const float4* const at = reinterpret_cast<const float4*>(x - off) + first + threadIdx.x;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int u = first + j * kThreads + int(threadIdx.x);
            if (u < last) {
                if (inner) {
                    const float4 w = __ldcs(at + j * kThreads);
                    v[j][0] = w.x, v[j][1] = w.y, v[j][2] = w.z, v[j][3] = w.w;
                } else {
                    load(u, v[j]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, v[j][e]);
        m = cta_reduce<true>(m, max_s);
        // of a part of -inf alone (and of the padding) nothing comes; a row of -inf alone gives NaN below
        const float base = m == -INFINITY ? 0.0f : m * h;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[j][e] = exp_of<H>(v[j][e], base, p);
                l += v[j][e];
            }
    } else {
        // A thread adds up to 65536 values: with what each addition rounds off kept beside the sum, or 8192 equal ones
        // would be off by 2^-13.  The base of the exponentials follows the maximum once that is 2^8 above, so a rising row
        // scales (and rounds) the sum a few times instead of at every unit.
        float lost = 0.0f, base = 0.0f;
        for (int u = first + threadIdx.x; u < last; u += kThreads) {
            load(u, v[0]);
            const float top = fmaxf(fmaxf(v[0][0], v[0][1]), fmaxf(v[0][2], v[0][3]));
            if (fmaf(top, h, -(m * h)) * p.k > 8.0f) {
                const float f = m == -INFINITY ? 0.0f : exp_of<H>(m, top * h, p);
                l *= f, lost *= f;
                m = top;
                base = m * h;
            }
            const float add = (exp_of<H>(v[0][0], base, p) + exp_of<H>(v[0][1], base, p)) +
                              (exp_of<H>(v[0][2], base, p) + exp_of<H>(v[0][3], base, p)) - lost;
            const float sum = l + add;
            lost = (sum - l) - add;
            l = sum;
        }
        const float top = cta_reduce<true>(m, max_s);
        l = m == -INFINITY ? l : l * factor<H>(m, top, p);  // (a NaN among -inf stays)
        m = top;
    }
    l = cta_reduce<false>(l, sum_s);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (int(threadIdx.x) < C) *cl.map_shared_rank(&part_s[rank], threadIdx.x) = make_float2(m, l);
    cl.sync();
    float top = -INFINITY, sum = 0.0f;
    for (int c = 0; c < C; ++c) top = fmaxf(top, part_s[c].x);
    for (int c = 0; c < C; ++c) sum += part_s[c].y == 0.0f ? 0.0f : part_s[c].y * factor<H>(part_s[c].x, top, p);
    if constexpr (NV > 0) {
        // a row of -inf alone: 0 / 0
        float4* const to = reinterpret_cast<float4*>(y - off) + first + threadIdx.x;
        const float f = (sum == 0.0f || m == -INFINITY ? 0.0f : factor<H>(m, top, p)) * (1.0f / sum);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int u = first + j * kThreads + int(threadIdx.x);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] *= f;
            if (inner) {
                if (u < last) *(to + j * kThreads) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
            } else if (u < last) {
                store(u, v[j]);
            }
        }
    } else {
        const float inv = 1.0f / sum, base = top == -INFINITY ? 0.0f : top * h;
        for (int u = first + threadIdx.x; u < last; u += kThreads) {
            load(u, v[0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[0][e] = exp_of<H>(v[0][e], base, p) * inv;
            store(u, v[0]);
        }
    }
}

template <int NV, bool H = false>
cudaError_t launch(const SoftmaxArgs& p, int64_t rows, int C, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows * C));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, softmax_kernel<NV, H>, p);
}

}  // namespace

cudaError_t launch_softmax(const float* x, float* y, int rows, int vocab, int64_t x_ld, int64_t y_ld, float scale,
                           int num_sms, cudaStream_t s)
{
    const bool halves = scale < 1e-36f;
    SoftmaxArgs p = {x, y, x_ld, y_ld, vocab, float(double(scale) * (halves ? 2 : 1) * 1.4426950408889634074), rows, 0};
    // the fewest CTAs that hold a row at 32 values per thread; more while SMs are idle and each has values left
    const bool whole = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && x_ld % 4 == 0;  // every row starts a unit
    const int64_t units = (int64_t(vocab) + (whole ? 3 : 6)) / 4;
    int C = 1;
    while (C < kMaxCluster && (units > int64_t(C) * kThreads * 8 || (int64_t(rows) * C * 2 <= num_sms && units > C * kThreads)))
        C *= 2;
    const int64_t per = ((units + C - 1) / C + kThreads - 1) / kThreads;  // units of a thread
    p.ahead = 2 * num_sms / C;
    if (halves) return launch<0, true>(p, rows, C, s);
    if (per <= 1) return launch<1>(p, rows, C, s);
    if (per <= 2) return launch<2>(p, rows, C, s);
    if (per <= 4) return launch<4>(p, rows, C, s);
    if (per <= 8) return launch<8>(p, rows, C, s);
    if (per <= 9) return launch<9>(p, rows, C, s);
    return launch<0>(p, rows, C, s);
}

}  // namespace mq
