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

// Tokens a sequence can have: positions and the ends of their tiles fit 32 bits.
__device__ __forceinline__ int64_t kv_capacity(const tq_kv4 &kv) {
    const int64_t c = kv.table_cols * kv.page_size;
    return c < 0x7fffff00 ? c : 0x7fffff00;
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

struct Geo {                                 // what the cutting of a batch depends on
    int g, causal, rows;                     // query heads a key/value head, mask, rows a row tile
    int64_t window;
};

struct Run {                                 // one row tile of one key/value head (at most 64 bytes)
    int b, h, rt;
    KvSeq q;
    int nrt;                                 // row tiles of the sequence
    int lo, hi, t0, cost;                    // positions its rows see, first tile, tiles (0: they see nothing)
};

// A row tile's positions and tiles of TILE positions.
template <int TILE>
__device__ __forceinline__ void range_of(const Geo &ge, const KvSeq &q, int rt, int &lo, int &hi, int &t0, int &cost) {
    const int rows = q.n * ge.g, r0 = rt * ge.rows;
    const int i0 = r0 / ge.g, i1 = (min(r0 + ge.rows, rows) - 1) / ge.g;
    const int p1 = q.len - q.n + i1;
    hi = p1 < 0 ? 0 : ge.causal ? min(p1 + 1, q.len) : q.len;
    const int64_t from = static_cast<int64_t>(q.len) - q.n + i0 - ge.window + 1;
    lo = ge.window > 0 && from > 0 ? static_cast<int>(from < hi ? from : hi) : 0;
    t0 = lo / TILE;
    cost = (hi + TILE - 1) / TILE - t0;
}

// Positions that row i of a sequence sees.
__device__ __forceinline__ void row_range(const Geo &ge, const KvSeq &q, int i, int &lo, int &hi) {
    const int pos = q.len - q.n + i;
    hi = pos < 0 ? 0 : ge.causal ? min(pos + 1, q.len) : q.len;
    const int64_t from = static_cast<int64_t>(pos) - ge.window + 1;
    lo = ge.window > 0 && from > 0 ? static_cast<int>(from < hi ? from : hi) : 0;
}

__device__ __forceinline__ int row_tiles(const Geo &ge, const KvSeq &q) {
    return (q.n * ge.g + ge.rows - 1) / ge.rows;
}

// The transform of a row held by eight neighbouring lanes, V neighbouring values
// each, scaled by sqrt(1 / (8 V)).
template <int V>
__device__ __forceinline__ void turn_row(float (&v)[V]) {
#pragma unroll
    for (int h = 1; h < V; h <<= 1)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(i & h)) {
                const float a = v[i], b = v[i + h];
                v[i] = a + b;
                v[i + h] = a - b;
            }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {
        const float sg = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(sg, v[i], __shfl_xor_sync(0xffffffffu, v[i], m));
    }
    const float c = sqrtf(1.0f / (8 * V));
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= c;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

__device__ __forceinline__ uint32_t bf16_bits2(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, uint64_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 2^k as fp32, k clamped to the normal range
__device__ __forceinline__ float pow2i(int k) {
    return __uint_as_float(static_cast<uint32_t>(min(max(k, -126), 127) + 127) << 23);
}

// a / b for a, b > 0: in 32 bits where they fit
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Zeros for the row tiles that see nothing (rows before position 0), a
// sequence a CTA.
template <int D>
__device__ __noinline__ static void zero_rows(const tq_kv4 &kv, const Kv4Attn &a, const Geo &ge) {
    for (int64_t b = blockIdx.x; b < kv.nseq; b += gridDim.x) {
        bool bad = false;
        const KvSeq q = kv_seq(kv, b, bad);
        const int none = q.n - q.len;        // rows before position 0
        if (none <= 0) continue;
        const int rows = q.n * ge.g, cut = q.len == 0 ? rows : none * ge.g / ge.rows * ge.rows;
        const int64_t pieces = static_cast<int64_t>(cut) * kv.heads * (D / 8);
        for (int64_t i = threadIdx.x; i < pieces; i += blockDim.x) {
            const int c = static_cast<int>(i % (D / 8));
            const int64_t k = i / (D / 8);
            const int row = static_cast<int>(k % cut), h = static_cast<int>(k / cut);
            const int64_t tok = q.start + row / ge.g;
            const int hq = h * ge.g + row % ge.g;
            *reinterpret_cast<uint4 *>(a.O + tok * a.ldo + static_cast<int64_t>(hq) * D + c * 8) = make_uint4(0, 0, 0, 0);
            if (a.lse && c == 0) a.lse[tok * a.heads_q + hq] = -INFINITY;
        }
    }
}

}  // namespace tq
