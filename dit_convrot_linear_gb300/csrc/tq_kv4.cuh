// Device helpers of the 4-bit cache: where a block of 16 tokens lies, and the
// checked reads of the batch's device arrays.
#pragma once

#include "tq_internal.cuh"

namespace tq {

constexpr int kKvBlock = 16;                                     // tokens a block

__host__ __device__ constexpr int kv_block_bytes(int dim) { return 16 * dim + 128; }

__host__ __device__ constexpr int64_t kv_record_bytes(int dim, int page_size) {
    return static_cast<int64_t>(page_size / kKvBlock) * kv_block_bytes(dim);
}

// A sequence of the batch: tokens in the cache, rows of this call, first row.
struct KvSeq {
    int len, n, start;
};

__device__ __forceinline__ int64_t kv_capacity(const tq_kv4 &kv) {
    const int64_t c = kv.table_cols * kv.page_size;
    return c < 0x7fffffff ? c : 0x7fffffff;
}

// Sequence b, its arrays checked: a length outside 0 .. capacity is taken as
// the nearest, a row range that is none as empty; `bad` is set for either.
__device__ __forceinline__ KvSeq kv_seq(const tq_kv4 &kv, int64_t b, bool &bad) {
    const int s = __ldg(kv.q_start + b), e = __ldg(kv.q_start + b + 1), l = __ldg(kv.kv_len + b);
    const int64_t cap = kv_capacity(kv);
    KvSeq q = {l, e - s, s};
    if (s < 0 || e < s || e > kv.tokens) {
        q.n = 0;
        q.start = 0;
        bad = true;
    }
    if (l < 0 || l > cap) {
        q.len = l < 0 ? 0 : static_cast<int>(cap);
        bad = true;
    }
    return q;
}

// The page of a sequence's token at `pos` (below its length), or -1.
__device__ __forceinline__ int kv_page(const tq_kv4 &kv, int64_t b, int pos) {
    const int page = __ldg(kv.table + b * kv.ldt + pos / kv.page_size);
    return page >= 0 && page < kv.npages ? page : -1;
}

// The number in the pool of the block that holds head h of a sequence's token
// at `pos`, or 2^32 - 1 (the host refuses pools of as many blocks).
__device__ __forceinline__ uint32_t kv_block_number(const tq_kv4 &kv, int64_t b, int h, int pos) {
    const int page = kv_page(kv, b, pos);
    const int per = kv.page_size / kKvBlock;
    return page < 0 ? 0xffffffffu
                    : (static_cast<uint32_t>(page) * kv.heads + h) * per + (pos & (kv.page_size - 1)) / kKvBlock;
}

// The block that holds head h of a page's token `slot`.
__device__ __forceinline__ unsigned char *kv_block(const tq_kv4 &kv, int page, int h, int slot) {
    const int64_t rec = kv_record_bytes(kv.dim, kv.page_size);
    return static_cast<unsigned char *>(kv.pool) + (static_cast<int64_t>(page) * kv.heads + h) * rec +
           (slot / kKvBlock) * kv_block_bytes(kv.dim);
}

}  // namespace tq
