// The product of 8-bit floating-point operands with a scale for each block of 128,
//   Y[m][n] = sum_b sx[b][m] * sw[n / 128][b] * sum_{k in block b} xq[m][k] * wq[n][k],
// of one matrix, or of one matrix an expert over rows sorted by expert.  The simple
// form: a CTA 64 x 64 outputs, a thread 4 x 4 of them in fp32.

#include <cuda_fp8.h>

#include "tq_internal.cuh"

namespace tq {
namespace {

constexpr int T = 64, KS = 32;

__device__ __forceinline__ float e4m3(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <typename OUT>
__global__ void __launch_bounds__(256) k_linear_f8(const F8Product p, unsigned int *status) {
    __shared__ float xs[KS][T + 1], ws[KS][T + 1];
    int64_t r0 = 0, r1 = p.M;
    if (p.offsets) {
        r0 = p.offsets[blockIdx.z];
        r1 = p.offsets[blockIdx.z + 1];
        int before = p.offsets[0];
        for (int e = 1; e < static_cast<int>(blockIdx.z); ++e) before = max(before, p.offsets[e]);
        if (r0 < 0 || r1 < r0 || r1 > p.M || r0 < before) {
            if (threadIdx.x == 0) atomicOr(status, kStatusIndex);
            return;
        }
    }
    const int64_t kb = (p.K + 127) / 128, nb = (p.N + 127) / 128;
    const uint8_t *W = p.Wq + static_cast<int64_t>(blockIdx.z) * p.N * p.K;
    const float *sw = p.sw + static_cast<int64_t>(blockIdx.z) * nb * kb;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * T;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t m0 = r0 + static_cast<int64_t>(blockIdx.y) * T; m0 < r1; m0 += static_cast<int64_t>(gridDim.y) * T) {
        float acc[4][4] = {};
        for (int64_t b = 0; b < kb; ++b) {
            float part[4][4] = {};
            for (int64_t k0 = b * 128; k0 < b * 128 + 128 && k0 < p.K; k0 += KS) {
                for (int i = threadIdx.x; i < T * KS; i += 256) {
                    const int r = i / KS, k = i % KS;
                    const bool in = k0 + k < p.K;
                    xs[k][r] = in && m0 + r < r1 ? e4m3(p.Xq[(m0 + r) * p.K + k0 + k]) : 0.0f;
                    ws[k][r] = in && n0 + r < p.N ? e4m3(W[(n0 + r) * p.K + k0 + k]) : 0.0f;
                }
                __syncthreads();
                for (int k = 0; k < KS; ++k)
                    for (int i = 0; i < 4; ++i)
                        for (int j = 0; j < 4; ++j)
                            part[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], part[i][j]);
                __syncthreads();
            }
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                    if (m < r1 && n < p.N)
                        acc[i][j] = fmaf(part[i][j], p.sx[b * p.M + m] * sw[n / 128 * kb + b], acc[i][j]);
                }
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m >= r1 || n >= p.N) continue;
                if constexpr (sizeof(OUT) == 4)
                    static_cast<float *>(p.Y)[m * p.ldy + n] = acc[i][j];
                else
                    static_cast<uint16_t *>(p.Y)[m * p.ldy + n] = f32_to_bf16_bits(acc[i][j]);
            }
    }
}

}  // namespace

size_t f8_workspace_bytes(const DeviceInfo &) { return 256; }

tq_status launch_linear_f8(const F8Product &p, const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    (void)dev;
    const int64_t gy = (p.M + T - 1) / T;
    const dim3 grid(static_cast<unsigned>((p.N + T - 1) / T), static_cast<unsigned>(gy < 1024 ? gy : 1024),
                    static_cast<unsigned>(p.offsets ? p.experts : 1));
    if (p.ytype == 0)
        k_linear_f8<float><<<grid, 256, 0, s>>>(p, status);
    else
        k_linear_f8<uint16_t><<<grid, 256, 0, s>>>(p, status);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace tq
