// mq_kv.cuh -- the paged key/value cache: its byte layout and the device-side
// lookups shared by the kernels that write it, read it and attend over it.
//
// A page holds kKvPage tokens of every key/value head, one block per head:
//   f16   K: head_dim/64 planes of [64 tokens][64 values] (128-byte rows), then V alike
//   q8_0  K codes [64 tokens][head_dim] (code + 128, one byte), V codes, then
//         the f16 scales of K [64][head_dim/32] and of V
// Within a row the 16-byte chunks are permuted by the token's row r (chunk c
// at c ^ swap(r)), so that the attention kernels read a block that a bulk
// copy brought into shared memory without bank conflicts; the f16 planes are
// exactly the 128-byte-swizzled tiles that tcgen05.mma reads, so an f16 block
// needs no pass over its values before the tensor cores take it.
// An element of a q8_0 cache stands for f16(scale * code): one rounding, which
// every reader makes, so all kernels see the same values.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "mq.h"

namespace mq {

constexpr int kKvPage = MQ_KV_PAGE_TOKENS;

// one (page, head) block, all sizes in bytes
template <int D, bool Q8>
struct KvBlock {
    static constexpr int kRow = Q8 ? D : 128;                 // bytes of a row (f16: of one 64-value plane)
    static constexpr int kVOff = kKvPage * D * (Q8 ? 1 : 2);  // V's first byte
    static constexpr int kScK = 2 * kKvPage * D;              // q8_0 only
    static constexpr int kScBytes = kKvPage * (D / 32) * 2;
    static constexpr int kBytes = Q8 ? 2 * kKvPage * D + 2 * kScBytes : 2 * kVOff;

    static __host__ __device__ constexpr int swap(int r) { return Q8 && D == 64 ? (r >> 1) & 3 : r & 7; }
    // byte of 16-byte chunk c (of a head's D values) of row r, from K's or V's first byte
    static __host__ __device__ constexpr int chunk(int r, int c)
    {
        return Q8 ? r * D + ((c ^ swap(r)) << 4) : (c >> 3) * (kKvPage * 128) + r * 128 + (((c & 7) ^ swap(r)) << 4);
    }
    static constexpr int kChunks = Q8 ? D / 16 : D / 8;  // 16-byte chunks of a row of D values
};

// the cache as the kernels take it
struct KvView {
    uint8_t* pages;
    const int32_t* table;
    int64_t n_pages;
    int32_t n_seqs, table_ld, n_kv_heads;
};

inline KvView kv_view(const mq_kv_cache& c)
{
    return KvView{static_cast<uint8_t*>(c.pages), c.table, c.n_pages, c.n_seqs, c.table_ld, c.n_kv_heads};
}

// two codes, each in the low byte of a half of magic 0x64 (1024 + code + 128),
// to f16(scale * code), scale as a pair: the subtraction is exact, the product rounds once
__device__ __forceinline__ uint32_t kv_pair(uint32_t u, uint32_t scale)
{
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tsub.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}"
        : "=r"(r)
        : "r"(u), "r"(0x64806480u), "r"(scale));  // 1024 + 128
    return r;
}

// one element of a block as fp32 (rare paths)
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

// first byte of the page that holds slot `slot` of sequence `seq`, as an
// offset into pages; -1 where the sequence, the slot or its page lies outside
// the cache (table entries are device data and are not trusted).
__device__ __forceinline__ int64_t kv_page_of(const KvView& c, int seq, int slot, int64_t page_bytes)
{
    if (seq < 0 || seq >= c.n_seqs || slot < 0 || slot / kKvPage >= c.table_ld) return -1;
    const int64_t p = __ldg(c.table + int64_t(seq) * c.table_ld + slot / kKvPage);
    return p < 0 || p >= c.n_pages ? -1 : p * page_bytes;
}

}  // namespace mq
