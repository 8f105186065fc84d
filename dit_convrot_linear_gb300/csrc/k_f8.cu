// Operands of the 8-bit floating-point product: e4m3 codes with a scale for each
// block of 128 columns of a row (activations) or of 128 rows and 128 columns
// (weights).
//
// A block's scale is the smallest power of two s = 2^j, j >= -126, for which
// |x| / s stays within e4m3's 448.  x / s is then exact (but for what e4m3 itself
// cannot hold), so a code is one rounding of x, and the value code * s needs none:
// a code of four exponent bits keeps the same relative precision wherever its
// block's largest value lies, so a finer scale would gain nothing.  No rotation
// for the same reason: a channel forty times its neighbours costs them no bits
// until they fall 2^13.8 below it (a block's largest |x| / s lies above 224, and e4m3's
// smallest normal number is 2^-6).
//
// Bound by memory: 2 B read (4 for the SwiGLU) and 1 B written a value.  A lane
// takes 16 columns (two 16-byte loads, one 16-byte store), eight lanes a block; eight
// CTAs an SM (32 registers) have the loads in flight that six (40) lack.  4032 rows of
// 12288: 24.6 us, 6040 GB/s (27.9 with six CTAs, 29.2 with a division for each piece of
// a row and the largest value sought among fp32 values); their SwiGLU 40.6, 6100 GB/s.
// Rows of four tokens' blocks a warp, for wider stores of the scales: 5% slower.
// 32768 rows of 2048 gathered from 4096: 28.9 us, half of it issue.

#include <cuda_fp8.h>

#include "tq_internal.cuh"

namespace tq {
namespace {

constexpr int kF8Warps = 8;                     // warps a CTA, each a row's 512 columns at a time

// Scale of a block by its largest |value| (fp32 bits): *inv = 1 / scale.
// A zero block: scale 0, codes 0.  Not finite: scale NaN, codes 0.
__device__ __forceinline__ float block_scale(uint32_t amax, float &inv) {
    if (amax == 0u) {
        inv = 0.0f;
        return 0.0f;
    }
    if (amax >= 0x7F800000u) {
        inv = 0.0f;
        return __uint_as_float(0x7FC00000u);
    }
    // 448 = 1.75 * 2^8: one binade more where the mantissa passes 1.75
    const int e = max(static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0), 1);
    inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// codes of 16 values; inv 0 (a block without a scale) gives zeros
__device__ __forceinline__ uint4 encode16(const float (&v)[16], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_e4m3(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    return inv == 0.0f ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void widen16(const uint4 &a, const uint4 &b, float (&v)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t amax16(const float (&v)[16]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// The same of packed bf16 values (their bits, without the sign, in the order of the values).
__device__ __forceinline__ uint32_t amax16_bf16(const uint4 &a, const uint4 &b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFF0000u, m << 16);
}

struct QuantF8 {
    const uint16_t *X, *U;         // U: the values are silu(X) * U
    int64_t ldx, ldu, M, K, rows_x;
    const int32_t *rows;           // source row of each row, or null
    uint8_t *Xq;
    float *sx;                     // [blocks][M]
    int chunks;                    // 512-column pieces of a row
    unsigned int *status;
};

template <bool SWIGLU>
__global__ void __launch_bounds__(32 * kF8Warps, 8) k_quant_act_f8(const QuantF8 p) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kF8Warps;
    const int64_t it = static_cast<int64_t>(blockIdx.x) * kF8Warps + (threadIdx.x >> 5);
    // (row and piece go on by what a step is in them: a division for each costs as much as the
    // loads)
    const int64_t rows = step / p.chunks;
    const int over = static_cast<int>(step - rows * p.chunks);
    int64_t m = it / p.chunks;
    for (int piece = static_cast<int>(it - m * p.chunks); m < p.M; m += rows, piece += over) {
        if (piece >= p.chunks) {
            piece -= p.chunks;
            if (++m >= p.M) break;
        }
        const int col = piece * 512 + lane * 16;
        int64_t src = m;
        if (p.rows) {
            src = p.rows[m];
            if (src < 0 || src >= p.rows_x) {
                if (src != -1 && lane == 0) atomicOr(p.status, kStatusIndex);
                continue;                          // left as it was
            }
        }
        const bool in = col < p.K;                 // K % 16 == 0: a lane's columns are all inside or all outside
        float v[16];
        uint32_t a = 0u;
        if (in) {
            const uint4 *x = reinterpret_cast<const uint4 *>(p.X + src * p.ldx + col);
            const uint4 x0 = __ldg(x), x1 = __ldg(x + 1);
            widen16(x0, x1, v);
            if constexpr (SWIGLU) {
                float u[16];
                const uint4 *y = reinterpret_cast<const uint4 *>(p.U + src * p.ldu + col);
                widen16(__ldg(y), __ldg(y + 1), u);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = silu_mul(v[i], u[i]);
                a = amax16(v);
            } else {
                a = amax16_bf16(x0, x1);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        float inv;
        const float s = block_scale(a, inv);
        if (in) {
            *reinterpret_cast<uint4 *>(p.Xq + m * p.K + col) = encode16(v, inv);
            if ((lane & 7) == 0) p.sx[static_cast<int64_t>(col >> 7) * p.M + m] = s;
        }
    }
}

// A CTA a 128 x 128 block of W, a thread 16 columns of every 32nd row.  Once a matrix, so
// left as it is: 12288 x 4096 37.7 us, 4000 GB/s; 2048 x 2048 5.8, 2160 GB/s (the launch).
__global__ void __launch_bounds__(256) k_quantize_weights_f8(const uint16_t *__restrict__ W, int64_t N, int64_t K,
                                                             int64_t ldw, uint8_t *__restrict__ codes,
                                                             float *__restrict__ scales, int kb) {
    __shared__ uint32_t part[8];
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / kb) * 128;
    const int k0 = static_cast<int>(blockIdx.x % kb) * 128;
    const int col = k0 + (threadIdx.x & 7) * 16;
    float v[4][16];
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + (threadIdx.x >> 3) + 32 * i;
        if (n < N && col < K) {
            const uint4 *x = reinterpret_cast<const uint4 *>(W + n * ldw + col);
            widen16(__ldg(x), __ldg(x + 1), v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] = 0.0f;
        }
        a = max(a, amax16(v[i]));
    }
    a = __reduce_max_sync(0xffffffffu, a);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, part[i]);
    float inv;
    const float s = block_scale(a, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + (threadIdx.x >> 3) + 32 * i;
        if (n < N && col < K) *reinterpret_cast<uint4 *>(codes + n * K + col) = encode16(v[i], inv);
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

}  // namespace

tq_status launch_quantize_weights_f8(const uint16_t *W, int64_t N, int64_t K, int64_t ldw, uint8_t *codes,
                                     float *scales, cudaStream_t s) {
    const int64_t kb = (K + 127) / 128, blocks = (N + 127) / 128 * kb;
    if (blocks > INT32_MAX) return TQ_ERR_OVERFLOW;
    k_quantize_weights_f8<<<static_cast<unsigned>(blocks), 256, 0, s>>>(W, N, K, ldw, codes, scales,
                                                                        static_cast<int>(kb));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

tq_status launch_quant_act_f8(const uint16_t *X, int64_t rows_x, int64_t K, int64_t ldx, const uint16_t *U,
                              int64_t ldu, const int32_t *rows, int64_t M, uint8_t *Xq, float *sx,
                              const DeviceInfo &dev, cudaStream_t s) {
    QuantF8 p{X, U, ldx, ldu, M, K, rows_x, rows, Xq, sx, static_cast<int>((K + 511) / 512), status_word()};
    if (!p.status) return TQ_ERR_DEVICE;
    const int64_t ctas = (M * p.chunks + kF8Warps - 1) / kF8Warps, most = static_cast<int64_t>(dev.sms) * 8;
    return launch_pdl(U ? k_quant_act_f8<true> : k_quant_act_f8<false>, static_cast<unsigned>(ctas < most ? ctas : most),
                      32 * kF8Warps, s, p);
}

}  // namespace tq
