// The 4-bit key/value cache: rows of keys and values rotated per head,
// quantised and put into their pages, and read back.  Memory: 2 B read and half
// a byte written per value, plus 4 B a row, and the converse.
//
// Prompts: a warp takes one block of 16 tokens of one head, keys or values.
// Four of the transform's index bits run on the tensor cores: a product with the
// 16 x 16 Hadamard matrix, exact in bf16, its sums of 16 in fp32; the others are
// butterflies between registers, a pair of values an instruction.  A lane holds
// the same 2 x dim / 4 values before and after: two tokens that share the cache's
// value words.  About 20 instructions a row (eight lanes a row, with three stages
// of shuffles, spend 85): 4132 tokens of 8 heads 7.9 us to append and 6.6 to read,
// 3.2 for their bytes; 32720 tokens 43.7 and 38.6, against 25.  What bounds them
// now is the loads in flight: 110 registers let two CTAs an SM.

#include <cfloat>

#include "tq_kv4.cuh"

namespace tq {
namespace {

constexpr int kSeqs = 512;                   // sequences looked at a time
constexpr int kCtas = 2;                     // CTAs an SM

// The sequences at hand: their blocks of this call's rows stand in a line.
struct Line {
    KvSeq q[kSeqs];
    int before[kSeqs + 1];                   // blocks of the sequences before
    int warp[kThreads / 32];
};

// First block of a sequence's rows (negative where it has more rows than
// tokens), and their number.
__device__ __forceinline__ int first_block(const KvSeq &q) { return (q.len - q.n) >> 4; }
__device__ __forceinline__ int blocks(const KvSeq &q) {
    return q.n > 0 ? (q.len >> 4) + ((q.len & 15) != 0) - first_block(q) : 0;
}

// Sequences `base` .. of the batch: the blocks of their rows.
__device__ __forceinline__ int line_up(const tq_kv4 &kv, int64_t base, Line &ln, bool &bad) {
    constexpr int EACH = kSeqs / kThreads;
    const int tid = threadIdx.x, lane = tid & 31;
    int own[EACH], sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int k = tid * EACH + i;
        own[i] = 0;
        if (base + k < kv.nseq) {
            const KvSeq q = kv_seq(kv, base + k, bad);
            ln.q[k] = q;
            own[i] = blocks(q);
        }
        sum += own[i];
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) ln.warp[tid >> 5] = x;
    __syncthreads();
    int at = x - sum, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < (tid >> 5)) at += ln.warp[w];
        all += ln.warp[w];
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        ln.before[tid * EACH + i] = at;
        at += own[i];
    }
    __syncthreads();
    return all;
}

// A warp's work: block `kb` of a sequence, one head, keys or values.  A lane's
// two rows are the tokens 16 kb + 2 g and the next, g = lane / 4.
struct Item {
    int64_t b, t[2];                         // sequence; rows of the call
    int h, kb;
    bool value, in, is[2];                   // keys or values; whether the block holds tokens, and rows of the call
};

__device__ __forceinline__ Item item_of(const tq_kv4 &kv, int64_t base, const Line &ln, int64_t w) {
    const int sides = 2 * kv.heads;
    const int64_t k = w / sides;
    const int j = static_cast<int>(w - k * sides);
    int lo = 0, hi = static_cast<int>(kv.nseq - base < kSeqs ? kv.nseq - base : kSeqs);
    while (hi - lo > 1) {                    // (the last of those that begin at k: the others are empty)
        const int mid = (lo + hi) >> 1;
        if (ln.before[mid] <= k) lo = mid;
        else hi = mid;
    }
    const KvSeq q = ln.q[lo];
    Item it;
    it.b = base + lo;
    it.value = j >= kv.heads;
    it.h = it.value ? j - kv.heads : j;
    it.kb = first_block(q) + static_cast<int>(k) - ln.before[lo];
    it.in = it.kb >= 0 && it.kb <= (q.len - 1) >> 4;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t i = static_cast<int64_t>(it.kb) * kKvBlock + 2 * ((threadIdx.x & 31) >> 2) + r - (q.len - q.n);
        it.is[r] = i >= 0 && i < q.n;
        it.t[r] = q.start + (it.is[r] ? i : 0);
    }
    return it;
}

// A row's scale from its largest rotated magnitude: NaN for a row that is not
// finite, so that it shows wherever the row is read.
__device__ __forceinline__ float scale_of(float amax) {
    return amax <= FLT_MAX ? __fdiv_rn(amax, 7.0f) : __uint_as_float(0x7FFFFFFFu);
}

// W words at p, aligned to them (up to 16 bytes)
template <int W>
__device__ __forceinline__ void store_words(unsigned char *p, const uint32_t *w) {
    if constexpr (W == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<uint4 *>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}

typedef unsigned long long pair_t;           // two fp32 values

__device__ __forceinline__ pair_t pair(float a, float b) {
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(pair_t r, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ void butterfly(pair_t &a, pair_t &b) {
    pair_t s, d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(s) : "l"(a), "l"(b));
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    a = s;
    b = d;
}

// d = a b, both rows of a lane: d[0], d[1] of the first, d[2], d[3] of the second
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// -1 to the power p, as bf16
__device__ __forceinline__ uint32_t sign(int p) { return p & 1 ? 0xBF80u : 0x3F80u; }

template <int D>
__global__ void __launch_bounds__(kThreads)
k_kv4_append(const __grid_constant__ tq_kv4 kv, const uint16_t *__restrict__ K, int64_t ldk,
             const uint16_t *__restrict__ V, int64_t ldv, unsigned int *status) {
    constexpr int CH = D / 32;                // pieces of 8 values a lane has of a row: CH j .., j = lane % 4
    __shared__ Line ln;
    const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    bool bad = false;
    pdl_launch_dependents();
    pdl_wait();
    // The matrix over index bits 0, 1 and j's: depth k = 2 j + e (+ 8 x) stands
    // for (j, x, e), column n for the same, so a sign is (-1)^(their common bits).
    const int pj = __popc(j & (g >> 1));
    const uint32_t b0 = sign(pj) | sign(pj + (g & 1)) << 16, b1 = b0 ^ 0x80008000u;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t base = 0; base < kv.nseq; base += kSeqs) {
        if (base) __syncthreads();
        bool off = false;                     // every CTA sees these: one's word is enough
        const int64_t all = static_cast<int64_t>(line_up(kv, base, ln, off)) * 2 * kv.heads;
        if (blockIdx.x == 0) bad |= off;
        for (int64_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < all; w += step) {
            const Item it = item_of(kv, base, ln, w);
            uint4 u[2][CH];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint16_t *src = (it.value ? V + it.t[r] * ldv : K + it.t[r] * ldk) + it.h * D + CH * 8 * j;
#pragma unroll
                for (int i = 0; i < CH; ++i) u[r][i] = it.is[r] ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
            }
            const int page = it.in ? kv_page(kv, it.b, it.kb * kKvBlock) : -1;
            if (it.in && page < 0) bad = true;
            // bits 0, 1 and j's; then bit 2 and the pieces'
            pair_t v[2][CH][2][2];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const uint32_t x[4] = {u[0][i].x, u[0][i].y, u[0][i].z, u[0][i].w};
                const uint32_t y[4] = {u[1][i].x, u[1][i].y, u[1][i].z, u[1][i].w};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float d[4];
                        mma0(d, x[2 * h], y[2 * h], x[2 * h + 1], y[2 * h + 1], b0, n ? b1 : b0);
                        v[0][i][h][n] = pair(d[0], d[1]);
                        v[1][i][h][n] = pair(d[2], d[3]);
                    }
            }
            const float cn = sqrtf(1.0f / D);
            uint32_t c[2][CH];
            float s[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n) butterfly(v[r][i][0][n], v[r][i][1][n]);
#pragma unroll
                for (int o = 1; o < CH; o <<= 1)
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        if (!(i & o))
#pragma unroll
                            for (int e = 0; e < 4; ++e) butterfly(v[r][i][e >> 1][e & 1], v[r][i + o][e >> 1][e & 1]);
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a, b;
                        split(v[r][i][e >> 1][e & 1], a, b);
                        amax = max_nan(amax, max_nan(fabsf(a), fabsf(b)));
                    }
                amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                s[r] = scale_of(amax * cn);
                // rint(v / s) as rint of the product with 1 / s, which is within
                // some units of 2^-24 of the quotient (nearer a tie than the
                // transform's own rounding); the sum with 1.5 2^23 + 8 rounds, and
                // leaves the code plus 8 in its low bits: their sum, each 16 times
                // the one before, is the word but for what the sums' high bits
                // come to.  The division itself where 1 / s is not a number.
                const float inv = s[r] > 0.0f ? cn * __frcp_rn(s[r]) : 0.0f;
                if (s[r] == 0.0f || (s[r] >= 1e-37f && s[r] <= FLT_MAX)) {
                    const pair_t k2 = pair(inv, inv), m2 = pair(12582920.0f, 12582920.0f);
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        uint32_t word = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pair_t q2;
                            asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q2) : "l"(v[r][i][e >> 1][e & 1]), "l"(k2), "l"(m2));
                            float a, b;
                            split(q2, a, b);
                            word += __float_as_uint(a) * (1u << (8 * e));
                            word += __float_as_uint(b) * (16u << (8 * e));
                        }
                        c[r][i] = word;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        c[r][i] = 0u;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float a, b;
                            split(v[r][i][e >> 2][(e >> 1) & 1], a, b);
                            const float x = (e & 1 ? b : a) * cn;
                            const int k = min(max(__float2int_rn(__fdiv_rn(x, s[r])), -7), 7);
                            c[r][i] |= static_cast<uint32_t>(k + 8) << (4 * e);
                        }
                    }
                }
            }
            if (page < 0) continue;
            unsigned char *blk = kv_block(kv, page, it.h, it.kb * kKvBlock & (kv.page_size - 1));
            if (!it.value) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (it.is[r]) store_words<CH>(blk + (2 * g + r) * (D / 2) + j * (D / 8), c[r]);
            } else {
                unsigned char *dst = blk + 8 * D + g * D + j * (D / 4);
                if (it.is[0] && it.is[1]) {
                    uint32_t o[2 * CH];
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        o[2 * i] = __byte_perm(c[0][i], c[1][i], 0x5410);
                        o[2 * i + 1] = __byte_perm(c[0][i], c[1][i], 0x7632);
                    }
                    store_words<2 * CH>(dst, o);
                } else {                     // the other halves belong to another call's token
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (it.is[r])
#pragma unroll
                            for (int i = 0; i < 2 * CH; ++i)
                                *reinterpret_cast<uint16_t *>(dst + 4 * i + 2 * r) =
                                    static_cast<uint16_t>(c[r][i / 2] >> (16 * (i % 2)));
                }
            }
            if (j < 2 && (j ? it.is[1] : it.is[0]))
                *reinterpret_cast<float *>(blk + 16 * D + (it.value ? 64 : 0) + 4 * (2 * g + j)) = j ? s[1] : s[0];
        }
    }
    if (bad) atomicOr(status, kStatusIndex);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
k_kv4_read(const __grid_constant__ tq_kv4 kv, uint16_t *__restrict__ K, int64_t ldk, uint16_t *__restrict__ V,
           int64_t ldv, unsigned int *status) {
    constexpr int CH = D / 32;                // pieces of 8 values a lane has of a row: j, j + 4 ..
    __shared__ Line ln;
    const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    bool bad = false;
    pdl_launch_dependents();
    pdl_wait();
    // The matrix over index bits 0, 2 and j's.  Nibbles four apart are an operand's
    // pair (e: bit 2, x: bit 0); a product's pair is bit 0, its two columns' bit 2.
    const int pj = __popc(j & (g >> 1)), en = g & 1;
    uint32_t m[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) m[n][x] = sign(pj + (x & en)) | sign(pj + (x & en) + n) << 16;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t base = 0; base < kv.nseq; base += kSeqs) {
        if (base) __syncthreads();
        bool off = false;
        const int64_t all = static_cast<int64_t>(line_up(kv, base, ln, off)) * 2 * kv.heads;
        if (blockIdx.x == 0) bad |= off;
        for (int64_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < all; w += step) {
            const Item it = item_of(kv, base, ln, w);
            uint16_t *out = it.value ? V : K;
            if (!out) continue;
            const int page = it.in ? kv_page(kv, it.b, it.kb * kKvBlock) : -1;
            if (it.in && page < 0) bad = true;
            uint32_t c[2][CH];
            float s[2] = {0.0f, 0.0f};        // (of a row that is not there, or has no page)
#pragma unroll
            for (int i = 0; i < CH; ++i) c[0][i] = c[1][i] = 0u;
            if (page >= 0) {
                const unsigned char *blk = kv_block(kv, page, it.h, it.kb * kKvBlock & (kv.page_size - 1));
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (it.is[r]) s[r] = *reinterpret_cast<const float *>(blk + 16 * D + (it.value ? 64 : 0) + 4 * (2 * g + r));
                if (!it.value) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int i = 0; i < CH; ++i)
                            c[r][i] = *reinterpret_cast<const uint32_t *>(blk + (2 * g + r) * (D / 2) + (4 * i + j) * 4);
                } else {
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const uint2 t = *reinterpret_cast<const uint2 *>(blk + 8 * D + g * D + (4 * i + j) * 8);
                        c[0][i] = __byte_perm(t.x, t.y, 0x5410);
                        c[1][i] = __byte_perm(t.x, t.y, 0x7632);
                    }
                }
            }
            // a nibble under 128's exponent is 128 plus it, and the code 136 less:
            // 136 D of the transform's first value
            pair_t v[2][CH][2][2];            // [row][piece][bit 1][bit 2], pairs of bit 0
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = ((c[e & 1][i] >> (4 * (2 * h + (e >> 1)))) & 0x000F000Fu) | 0x43004300u;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float d[4];
                        mma0(d, a[0], a[1], a[2], a[3], m[n][0], m[n][1]);
                        v[0][i][h][n] = pair(d[0], d[1]);
                        v[1][i][h][n] = pair(d[2], d[3]);
                    }
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n) butterfly(v[r][i][0][n], v[r][i][1][n]);
#pragma unroll
                for (int o = 1; o < CH; o <<= 1)
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        if (!(i & o))
#pragma unroll
                            for (int e = 0; e < 4; ++e) butterfly(v[r][i][e >> 1][e & 1], v[r][i + o][e >> 1][e & 1]);
                if (j == 0) {
                    float a, b;
                    split(v[r][0][0][0], a, b);
                    v[r][0][0][0] = pair(a - 136.0f * D, b);
                }
                if (!it.is[r]) continue;
                const float f = s[r] == 0.0f ? 0.0f : s[r] * sqrtf(1.0f / D);
                uint16_t *dst = out + it.t[r] * (it.value ? ldv : ldk) + it.h * D + 8 * j;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {            // values 2 e and 2 e + 1
                        float a, b;
                        split(v[r][i][e & 1][e >> 1], a, b);
                        o[e] = bf16_bits2(a * f, b * f);
                    }
                    *reinterpret_cast<uint4 *>(dst + 32 * i) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
    if (bad) atomicOr(status, kStatusIndex);
}

// ---------------------------------------------------------------- few rows
// A row apart, eight lanes each: the search for its sequence is all there is
// before its values, and no lane waits for the fifteen rows beside it.

constexpr int kLanes = 8;                    // lanes a row
constexpr int kRows = 32 / kLanes;           // rows a warp
constexpr int kStarts = 1024;                // row ranges held in shared memory

// The sequence that owns row t (row ranges run forwards; -1: none), and its
// description.  `starts` holds q_start in shared memory where it fits.
__device__ __forceinline__ int64_t owner_of(const tq_kv4 &kv, const int *starts, int64_t t, KvSeq &q, bool &bad) {
    const bool near = kv.nseq <= kStarts;
    int64_t lo = 0, hi = kv.nseq;          // last b with q_start[b] <= t lies in [lo, hi)
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if ((near ? starts[mid] : __ldg(kv.q_start + mid)) <= t) lo = mid;
        else hi = mid;
    }
    q = kv_seq(kv, lo, bad);
    return t >= q.start && t < static_cast<int64_t>(q.start) + q.n ? lo : -1;
}

// q_start into shared memory, and every sequence's arrays checked by one CTA.
__device__ __forceinline__ void begin(const tq_kv4 &kv, int *starts, bool &bad) {
    if (kv.nseq <= kStarts)
        for (int64_t b = threadIdx.x; b < kv.nseq; b += kThreads) starts[b] = __ldg(kv.q_start + b);
    if (blockIdx.x == 0)
        for (int64_t b = threadIdx.x; b < kv.nseq; b += kThreads) kv_seq(kv, b, bad);
    __syncthreads();
}

// A lane's work: row t of head h, keys or values.  Items run over four tokens,
// then heads and sides, then the next tokens.
struct Row {
    int64_t t;
    int h;
    bool value, is;
};

__device__ __forceinline__ Row row_of(const tq_kv4 &kv, int64_t w) {
    const int sides = 2 * kv.heads;
    const int64_t four = w / sides;
    const int j = static_cast<int>(w - four * sides);
    Row it;
    it.t = four * kRows + (threadIdx.x & 31) / kLanes;
    it.value = j >= kv.heads;
    it.h = it.value ? j - kv.heads : j;
    it.is = it.t < kv.tokens;
    return it;
}

__device__ __forceinline__ int64_t warps_of(const tq_kv4 &kv) { return (kv.tokens + kRows - 1) / kRows * 2 * kv.heads; }

// B bytes at p
template <int B>
__device__ __forceinline__ void store_bytes(unsigned char *p, const uint32_t *w) {
    if constexpr (B == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (B == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p) = w[0];
}

template <int D>
__global__ void __launch_bounds__(kThreads)
k_kv4_append_rows(const __grid_constant__ tq_kv4 kv, const uint16_t *__restrict__ K, int64_t ldk,
             const uint16_t *__restrict__ V, int64_t ldv, unsigned int *status) {
    constexpr int N = D / kLanes;             // values a lane
    __shared__ int starts[kStarts];
    const int lane = threadIdx.x & 31, l8 = lane % kLanes;
    bool bad = false;
    pdl_launch_dependents();
    pdl_wait();
    begin(kv, starts, bad);
    const int64_t all = warps_of(kv);
    for (int64_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < all;
         w += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const Row it = row_of(kv, w);
        float v[N];
        {
            const uint16_t *src = (it.value ? V + (it.is ? it.t : 0) * ldv : K + (it.is ? it.t : 0) * ldk) + it.h * D + l8 * N;
#pragma unroll
            for (int i = 0; i < N; i += 8) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src + i));
                const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[i + 2 * e] = __uint_as_float(x[e] << 16);
                    v[i + 2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
                }
            }
        }
        KvSeq q;
        const int64_t b = owner_of(kv, starts, it.is ? it.t : 0, q, bad);
        const int64_t pos = b < 0 || !it.is ? -1 : q.len - q.n + (it.t - q.start);
        const int page = pos < 0 ? -1 : kv_page(kv, b, static_cast<int>(pos));
        if (pos >= 0 && page < 0) bad = true;
        const bool keep = page >= 0;
        turn_row<N>(v);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) amax = max_nan(amax, fabsf(v[i]));
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const float s = scale_of(amax);
        // rint(v / s) as rint of the product with 1 / s, which is within three
        // units of 2^-24 of the quotient (nearer a tie than the transform's own
        // rounding); the sum with 1.5 2^23 + 8 rounds, and leaves the code plus 8
        // in its low bits.  The division itself where 1 / s is not a number.
        const float r = __frcp_rn(s);
        uint32_t c[N / 8];
#pragma unroll
        for (int i = 0; i < N / 8; ++i) c[i] = 0u;
        if (s >= 1e-37f) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                c[i / 8] |= (__float_as_uint(fmaf(v[i], r, 12582920.0f)) & 15u) << (4 * (i % 8));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int k = s == 0.0f ? 0 : min(max(__float2int_rn(__fdiv_rn(v[i], s)), -7), 7);
                c[i / 8] |= static_cast<uint32_t>(k + 8) << (4 * (i % 8));
            }
        }
        const int slot = static_cast<int>(pos & (kv.page_size - 1)), row = slot % kKvBlock;
        unsigned char *blk = keep ? kv_block(kv, page, it.h, slot) : nullptr;
        if (!it.value) {
            if (keep) store_bytes<N / 2>(blk + row * (D / 2) + l8 * (N / 2), c);
        } else {
            // two bytes of every four are this token's; where the next group of
            // lanes holds the token that the others belong to, the two share
            // the words: the even token's lanes write the first half of them
            const uint64_t mine = keep ? reinterpret_cast<uint64_t>(blk) + (row >> 1) * D : 0;
            const uint64_t other = __shfl_xor_sync(0xffffffffu, mine, kLanes);
            const bool odd = row & 1, late = (lane / kLanes) & 1;
            const bool both = keep && mine == other && odd == late;
            uint32_t x[N / 8];
#pragma unroll
            for (int i = 0; i < N / 8; ++i) x[i] = __shfl_xor_sync(0xffffffffu, c[i], kLanes);
            unsigned char *dst = blk + 8 * D + (row >> 1) * D + l8 * N;
            if (both) {
                uint32_t o[N / 4];
#pragma unroll
                for (int i = 0; i < N / 8; ++i) {
                    const uint32_t ev = odd ? x[i] : c[i], od = odd ? c[i] : x[i];
                    o[2 * i] = __byte_perm(ev, od, 0x5410);
                    o[2 * i + 1] = __byte_perm(ev, od, 0x7632);
                }
                constexpr int H = N / 8;                 // words a lane writes
                uint32_t h[H];
#pragma unroll
                for (int i = 0; i < H; ++i) h[i] = odd ? o[H + i] : o[i];
                store_bytes<4 * H>(dst + (odd ? 4 * H : 0), h);
            } else if (keep) {
#pragma unroll
                for (int i = 0; i < N / 4; ++i)
                    *reinterpret_cast<uint16_t *>(dst + 4 * i + (odd ? 2 : 0)) =
                        static_cast<uint16_t>(c[i / 2] >> (16 * (i % 2)));
            }
        }
        if (keep && l8 == 0) *reinterpret_cast<float *>(blk + 16 * D + (it.value ? 64 : 0) + 4 * row) = s;
    }
    if (bad) atomicOr(status, kStatusIndex);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
k_kv4_read_rows(const __grid_constant__ tq_kv4 kv, uint16_t *__restrict__ K, int64_t ldk, uint16_t *__restrict__ V,
           int64_t ldv, unsigned int *status) {
    constexpr int N = D / kLanes;
    __shared__ int starts[kStarts];
    const int l8 = (threadIdx.x & 31) % kLanes;
    bool bad = false;
    pdl_launch_dependents();
    pdl_wait();
    begin(kv, starts, bad);
    const int64_t all = warps_of(kv);
    for (int64_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < all;
         w += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const Row it = row_of(kv, w);
        uint16_t *out = it.value ? V : K;
        if (!out) continue;                              // the warp's items are of one side
        KvSeq q;
        const int64_t b = owner_of(kv, starts, it.is ? it.t : 0, q, bad);
        const bool owned = it.is && b >= 0;
        const int64_t pos = owned ? q.len - q.n + (it.t - q.start) : -1;
        const int page = pos < 0 ? -1 : kv_page(kv, b, static_cast<int>(pos));
        if (pos >= 0 && page < 0) bad = true;
        uint32_t c[N / 8];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N / 8; ++i) c[i] = 0x88888888u;
        if (page >= 0) {
            const int slot = static_cast<int>(pos & (kv.page_size - 1)), row = slot % kKvBlock;
            const unsigned char *blk = kv_block(kv, page, it.h, slot);
            s = *reinterpret_cast<const float *>(blk + 16 * D + (it.value ? 64 : 0) + 4 * row);
            if (!it.value) {
                const uint32_t *src = reinterpret_cast<const uint32_t *>(blk + row * (D / 2) + l8 * (N / 2));
#pragma unroll
                for (int i = 0; i < N / 8; ++i) c[i] = src[i];
            } else {                                     // both tokens' words, one's halves
                const uint2 *src = reinterpret_cast<const uint2 *>(blk + 8 * D + (row >> 1) * D + l8 * N);
                const uint32_t pick = row & 1 ? 0x7632u : 0x5410u;
#pragma unroll
                for (int i = 0; i < N / 8; ++i) {
                    const uint2 u = src[i];
                    c[i] = __byte_perm(u.x, u.y, pick);
                }
            }
        }
        // a nibble under 2^23's exponent is 2^23 plus it; the code is 8 less
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = (__uint_as_float(0x4B000000u | ((c[i / 8] >> (4 * (i % 8))) & 15u)) - 8388616.0f) * s;
        turn_row<N>(v);
        if (!owned) continue;
        uint32_t o[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        uint16_t *dst = out + it.t * (it.value ? ldv : ldk) + it.h * D + l8 * N;
#pragma unroll
        for (int i = 0; i < N / 2; i += 4)
            *reinterpret_cast<uint4 *>(dst + 2 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
    if (bad) atomicOr(status, kStatusIndex);
}

constexpr int kRowCtas = 8;                  // CTAs an SM

int64_t row_warps(const tq_kv4 &kv) { return (kv.tokens + kRows - 1) / kRows * 2 * kv.heads; }

// Blocks of the call's rows at most: each has a row, and but for two of a
// sequence sixteen.
int64_t block_warps(const tq_kv4 &kv) {
    const int64_t most = kv.tokens / kKvBlock + 2 * kv.nseq;
    return (kv.tokens < most ? kv.tokens : most) * 2 * kv.heads;
}

// Rows are taken on their own while their warps, four rows each, are no more
// than the schedulers hold at once: 64 decoded tokens of 8 heads 3.5 us to
// append and 3.2 to read, against 4.6 and 3.8 by blocks; 2048 rows of 2 heads
// alike either way; 8192 of 8 heads 24 and 23 against 15 and 13.
bool few_rows(const tq_kv4 &kv, const DeviceInfo &dev) { return row_warps(kv) <= 16 * static_cast<int64_t>(dev.sms); }

template <typename F, typename... A>
tq_status launch_warps(F kern, int64_t warps, int64_t ctas, const tq_kv4 &kv, const DeviceInfo &dev, cudaStream_t s, A... args) {
    const int64_t want = (warps + kThreads / 32 - 1) / (kThreads / 32), room = dev.sms * ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < room ? want : room));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, kv, args...);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace

tq_status launch_kv4_append(const tq_kv4 &kv, const uint16_t *K, int64_t ldk, const uint16_t *V, int64_t ldv,
                            const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    if (few_rows(kv, dev)) {
        auto kern = kv.dim == 64 ? k_kv4_append_rows<64> : kv.dim == 128 ? k_kv4_append_rows<128> : k_kv4_append_rows<256>;
        return launch_warps(kern, row_warps(kv), kRowCtas, kv, dev, s, K, ldk, V, ldv, status);
    }
    auto kern = kv.dim == 64 ? k_kv4_append<64> : kv.dim == 128 ? k_kv4_append<128> : k_kv4_append<256>;
    return launch_warps(kern, block_warps(kv), kCtas, kv, dev, s, K, ldk, V, ldv, status);
}

tq_status launch_kv4_read(const tq_kv4 &kv, uint16_t *K, int64_t ldk, uint16_t *V, int64_t ldv,
                          const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    if (few_rows(kv, dev)) {
        auto kern = kv.dim == 64 ? k_kv4_read_rows<64> : kv.dim == 128 ? k_kv4_read_rows<128> : k_kv4_read_rows<256>;
        return launch_warps(kern, row_warps(kv), kRowCtas, kv, dev, s, K, ldk, V, ldv, status);
    }
    auto kern = kv.dim == 64 ? k_kv4_read<64> : kv.dim == 128 ? k_kv4_read<128> : k_kv4_read<256>;
    return launch_warps(kern, block_warps(kv), kCtas, kv, dev, s, K, ldk, V, ldv, status);
}

}  // namespace tq
