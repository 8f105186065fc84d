// The 4-bit key/value cache: rows of keys and values rotated per head,
// quantised and put into their pages, and read back.
//
// Eight lanes take one head's row of keys or of values, dim / 8 neighbouring
// values each, and a warp four tokens of the same head.  The butterfly runs
// inside a lane but for three of its stages (a warp per row, as the projections'
// rotation has it, spent 250 instructions a row, most of them shuffles: 33 us
// for 8 K tokens of 8 heads, against 3 us for its bytes).  Memory: 2 B read and
// half a byte written per value, plus 4 B a row, and the converse.

#include "tq_kv4.cuh"

namespace tq {
namespace {

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
struct Item {
    int64_t t;
    int h;
    bool value, is;
};

__device__ __forceinline__ Item item_of(const tq_kv4 &kv, int64_t w) {
    const int sides = 2 * kv.heads;
    const int64_t four = w / sides;
    const int j = static_cast<int>(w - four * sides);
    Item it;
    it.t = four * kRows + (threadIdx.x & 31) / kLanes;
    it.value = j >= kv.heads;
    it.h = it.value ? j - kv.heads : j;
    it.is = it.t < kv.tokens;
    return it;
}

__device__ __forceinline__ int64_t items(const tq_kv4 &kv) { return (kv.tokens + kRows - 1) / kRows * 2 * kv.heads; }

// E / 2 words of 16 bytes or fewer at p
template <int B>
__device__ __forceinline__ void store_bytes(unsigned char *p, const uint32_t *w) {
    if constexpr (B == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (B == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p) = w[0];
}

template <int D>
__global__ void __launch_bounds__(kThreads)
k_kv4_append(const __grid_constant__ tq_kv4 kv, const uint16_t *__restrict__ K, int64_t ldk,
             const uint16_t *__restrict__ V, int64_t ldv, unsigned int *status) {
    constexpr int N = D / kLanes;             // values a lane
    __shared__ int starts[kStarts];
    const int lane = threadIdx.x & 31, l8 = lane % kLanes;
    bool bad = false;
    pdl_launch_dependents();
    pdl_wait();
    begin(kv, starts, bad);
    const int64_t all = items(kv);
    for (int64_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < all;
         w += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const Item it = item_of(kv, w);
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
        for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const float s = __fdiv_rn(amax, 7.0f);
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
k_kv4_read(const __grid_constant__ tq_kv4 kv, uint16_t *__restrict__ K, int64_t ldk, uint16_t *__restrict__ V,
           int64_t ldv, unsigned int *status) {
    constexpr int N = D / kLanes;
    __shared__ int starts[kStarts];
    const int l8 = (threadIdx.x & 31) % kLanes;
    bool bad = false;
    pdl_launch_dependents();
    pdl_wait();
    begin(kv, starts, bad);
    const int64_t all = items(kv);
    for (int64_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < all;
         w += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const Item it = item_of(kv, w);
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

template <typename F, typename... A>
tq_status launch_rows(F kern, const tq_kv4 &kv, const DeviceInfo &dev, cudaStream_t s, A... args) {
    const int64_t want = ((kv.tokens + kRows - 1) / kRows * 2 * kv.heads + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = static_cast<int64_t>(dev.sms) * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
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
    auto kern = kv.dim == 64 ? k_kv4_append<64> : kv.dim == 128 ? k_kv4_append<128> : k_kv4_append<256>;
    return launch_rows(kern, kv, dev, s, K, ldk, V, ldv, status);
}

tq_status launch_kv4_read(const tq_kv4 &kv, uint16_t *K, int64_t ldk, uint16_t *V, int64_t ldv,
                          const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    auto kern = kv.dim == 64 ? k_kv4_read<64> : kv.dim == 128 ? k_kv4_read<128> : k_kv4_read<256>;
    return launch_rows(kern, kv, dev, s, K, ldk, V, ldv, status);
}

}  // namespace tq
