// The 4-bit key/value cache: rows of keys and values rotated per head,
// quantised and put into their pages, and read back.
//
// A warp takes one head's row of keys or of values: dim / 32 values a lane, the
// butterfly of the projections' rotation (scaled by sqrt(1 / dim)), the row's
// largest magnitude, s = fp32(amax / 7), codes by IEEE division.  Both kernels
// are bound by memory: 2 B read and half a byte written per value, plus 4 B a
// row, and the converse.

#include "tq_kv4.cuh"

namespace tq {
namespace {

// The sequence that owns row t (row ranges run forwards; -1: none), and its
// description.
__device__ __forceinline__ int64_t owner_of(const tq_kv4 &kv, int64_t t, KvSeq &q, bool &bad) {
    int64_t lo = 0, hi = kv.nseq;          // last b with q_start[b] <= t lies in [lo, hi)
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(kv.q_start + mid) <= t) lo = mid;
        else hi = mid;
    }
    q = kv_seq(kv, lo, bad);
    return t >= q.start && t < static_cast<int64_t>(q.start) + q.n ? lo : -1;
}

// byte offset, inside a block, of lane values [lane * E, lane * E + E) of the
// token at row r: for E = 2 one byte, for E = 4 two, for E = 8 four (keys) or
// twice two, 4 bytes apart (values)
template <int E>
__device__ __forceinline__ int codes_at(bool value, int r, int lane) {
    constexpr int D = 32 * E;
    if (!value) return r * (D / 2) + lane * E / 2;
    const int base = 8 * D + (r >> 1) * D + (r & 1) * 2;
    return E == 2 ? base + (lane >> 1) * 4 + (lane & 1) : base + lane * E;
}

template <int E>
__global__ void __launch_bounds__(kThreads)
k_kv4_append(const __grid_constant__ tq_kv4 kv, const uint16_t *__restrict__ K, int64_t ldk,
             const uint16_t *__restrict__ V, int64_t ldv, unsigned int *status) {
    constexpr int D = 32 * E;
    const int lane = threadIdx.x & 31;
    const int64_t rows = kv.tokens * kv.heads * 2;
    bool bad = false;
    if (blockIdx.x == 0)                   // every sequence's arrays, once a call
        for (int64_t b = threadIdx.x; b < kv.nseq; b += kThreads) kv_seq(kv, b, bad);
    for (int64_t i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < rows;
         i += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const int64_t t = i / (2 * kv.heads);
        const int j = static_cast<int>(i - t * 2 * kv.heads);
        const bool value = j >= kv.heads;
        const int h = value ? j - kv.heads : j;
        float v[8];
        load_bf16<E, float>((value ? V + t * ldv : K + t * ldk) + h * D + lane * E, v);
        KvSeq q;
        const int64_t b = owner_of(kv, t, q, bad);
        const int64_t pos = b < 0 ? -1 : q.len - q.n + (t - q.start);
        if (pos < 0) continue;
        const int page = kv_page(kv, b, static_cast<int>(pos));
        if (page < 0) {
            bad = true;
            continue;
        }
        warp_fwht<E, float>(v);
        const float c = sqrtf(1.0f / D);
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[e] = c * v[e];
            amax = fmaxf(amax, fabsf(v[e]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float s = __fdiv_rn(amax, 7.0f);
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int code = s == 0.0f ? 0 : min(max(__float2int_rn(__fdiv_rn(v[e], s)), -7), 7);
            w |= static_cast<uint32_t>(code + 8) << (4 * e);
        }
        const int slot = static_cast<int>(pos % kv.page_size), r = slot % kKvBlock;
        unsigned char *blk = kv_block(kv, page, h, slot);
        unsigned char *dst = blk + codes_at<E>(value, r, lane);
        if constexpr (E == 2) {
            *dst = static_cast<unsigned char>(w);
        } else if constexpr (E == 4) {
            *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(w);
        } else if (value) {
            *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(w);
            *reinterpret_cast<uint16_t *>(dst + 4) = static_cast<uint16_t>(w >> 16);
        } else {
            *reinterpret_cast<uint32_t *>(dst) = w;
        }
        if (lane == 0) *reinterpret_cast<float *>(blk + 16 * D + (value ? 64 : 0) + 4 * r) = s;
    }
    if (bad) atomicOr(status, kStatusIndex);
}

template <int E>
__global__ void __launch_bounds__(kThreads)
k_kv4_read(const __grid_constant__ tq_kv4 kv, uint16_t *__restrict__ K, int64_t ldk, uint16_t *__restrict__ V,
           int64_t ldv, unsigned int *status) {
    constexpr int D = 32 * E;
    const int lane = threadIdx.x & 31;
    const int64_t rows = kv.tokens * kv.heads * 2;
    bool bad = false;
    if (blockIdx.x == 0)
        for (int64_t b = threadIdx.x; b < kv.nseq; b += kThreads) kv_seq(kv, b, bad);
    for (int64_t i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < rows;
         i += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const int64_t t = i / (2 * kv.heads);
        const int j = static_cast<int>(i - t * 2 * kv.heads);
        const bool value = j >= kv.heads;
        const int h = value ? j - kv.heads : j;
        uint16_t *out = value ? V : K;
        if (!out) continue;
        out += t * (value ? ldv : ldk) + h * D + lane * E;
        KvSeq q;
        const int64_t b = owner_of(kv, t, q, bad);
        if (b < 0) continue;
        const int64_t pos = q.len - q.n + (t - q.start);
        const int page = pos < 0 ? -1 : kv_page(kv, b, static_cast<int>(pos));
        if (pos >= 0 && page < 0) bad = true;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        if (page >= 0) {
            const int slot = static_cast<int>(pos % kv.page_size), r = slot % kKvBlock;
            const unsigned char *blk = kv_block(kv, page, h, slot);
            const unsigned char *src = blk + codes_at<E>(value, r, lane);
            uint32_t w;
            if constexpr (E == 2) {
                w = *src;
            } else if constexpr (E == 4) {
                w = *reinterpret_cast<const uint16_t *>(src);
            } else if (value) {
                w = *reinterpret_cast<const uint16_t *>(src) |
                    (static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(src + 4)) << 16);
            } else {
                w = *reinterpret_cast<const uint32_t *>(src);
            }
            const float s = *reinterpret_cast<const float *>(blk + 16 * D + (value ? 64 : 0) + 4 * r);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = static_cast<float>(static_cast<int>((w >> (4 * e)) & 15u) - 8) * s;
            warp_fwht<E, float>(v);
            const float c = sqrtf(1.0f / D);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = c * v[e];
        }
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            p[e] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * e])) |
                   (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * e + 1])) << 16);
        if constexpr (E == 8) *reinterpret_cast<uint4 *>(out) = make_uint4(p[0], p[1], p[2], p[3]);
        else if constexpr (E == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(p[0], p[1]);
        else *reinterpret_cast<uint32_t *>(out) = p[0];
    }
    if (bad) atomicOr(status, kStatusIndex);
}

unsigned row_blocks(const tq_kv4 &kv, const DeviceInfo &dev) {
    const int64_t want = (kv.tokens * kv.heads * 2 + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = static_cast<int64_t>(dev.sms) * 8 * 4;
    return static_cast<unsigned>(want < most ? want : most);
}

}  // namespace

tq_status launch_kv4_append(const tq_kv4 &kv, const uint16_t *K, int64_t ldk, const uint16_t *V, int64_t ldv,
                            const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    auto kern = kv.dim == 64 ? k_kv4_append<2> : kv.dim == 128 ? k_kv4_append<4> : k_kv4_append<8>;
    kern<<<row_blocks(kv, dev), kThreads, 0, s>>>(kv, K, ldk, V, ldv, status);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

tq_status launch_kv4_read(const tq_kv4 &kv, uint16_t *K, int64_t ldk, uint16_t *V, int64_t ldv,
                          const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    auto kern = kv.dim == 64 ? k_kv4_read<2> : kv.dim == 128 ? k_kv4_read<4> : k_kv4_read<8>;
    kern<<<row_blocks(kv, dev), kThreads, 0, s>>>(kv, K, ldk, V, ldv, status);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace tq
