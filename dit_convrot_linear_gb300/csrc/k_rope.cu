// Rotary positions with one or more axes (Su et al., "RoFormer", 2021): pair p
// of every head of token t turns by the angle pos[axis(p)][t] * inv_freq[p].
//
// Memory-bound: 2 B read and 2 B written per value; a token's sines and
// cosines are formed once and shared by its heads.

#include <string.h>

#include "tq_internal.cuh"

namespace tq {
namespace {

struct RopeParams {
    const uint16_t *X;
    uint16_t *Y;
    int64_t T, ldx, ldy;
    const int32_t *pos;
    int64_t ldpos;
    const float *inv_freq;
    int heads, dim, pairs, interleaved;
    uint8_t axis[TQ_ROPE_MAX_DIM / 2];
};

// cos and sin of pos * f.  The product of an int32 and an fp32 number is exact
// in fp64 (31 + 24 bits, rounded once to 53), and one multiple of 2 pi (in two
// parts) taken off it in fp64 leaves an argument within [-pi, pi] whose error
// stays below 2^-40 for every int32 position.
__device__ __forceinline__ float2 turn_of(int32_t pos, float f) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    constexpr double kTwoPiLow = 2.4492935982947064e-16;   // 2 pi - kTwoPi
    const double a = static_cast<double>(pos) * static_cast<double>(f);
    const double k = rint(a * (1.0 / kTwoPi));
    const double r = fma(-k, kTwoPiLow, fma(-k, kTwoPi, a));
    float s, c;
    sincosf(static_cast<float>(r), &s, &c);
    return make_float2(c, s);
}

__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[TQ_ROPE_MAX_DIM / 2];
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        __syncthreads();
        for (int i = threadIdx.x; i < p.pairs; i += kThreads)
            cs[i] = turn_of(__ldg(p.pos + p.axis[i] * p.ldpos + t), __ldg(p.inv_freq + i));
        __syncthreads();
        const uint16_t *x = p.X + t * p.ldx;
        uint16_t *y = p.Y + t * p.ldy;
        // one pair a step; then the values past the pairs, copied
        const int rest = p.dim - 2 * p.pairs;
        const int step = p.interleaved ? 1 : p.pairs;
        for (int i = threadIdx.x; i < p.heads * p.pairs; i += kThreads) {
            const int h = i / p.pairs, q = i - h * p.pairs;
            const int64_t at = static_cast<int64_t>(h) * p.dim + (p.interleaved ? 2 * q : q);
            const float a = bf16_bits_to_f32(x[at]), b = bf16_bits_to_f32(x[at + step]);
            const float2 w = cs[q];
            y[at] = f32_to_bf16_bits(a * w.x - b * w.y);
            y[at + step] = f32_to_bf16_bits(b * w.x + a * w.y);
        }
        if (p.X == p.Y) continue;
        for (int i = threadIdx.x; i < p.heads * rest; i += kThreads) {
            const int h = i / rest;
            const int64_t at = static_cast<int64_t>(h) * p.dim + 2 * p.pairs + (i - h * rest);
            y[at] = x[at];
        }
    }
}

}  // namespace

tq_status launch_rope(const uint16_t *X, int64_t T, int heads, int dim, int64_t ldx, const tq_rope_spec &spec,
                      uint16_t *Y, int64_t ldy, const DeviceInfo &dev, cudaStream_t s) {
    RopeParams p;
    memset(&p, 0, sizeof(p));
    p.X = X;
    p.Y = Y;
    p.T = T;
    p.ldx = ldx;
    p.ldy = ldy;
    p.pos = spec.pos;
    p.ldpos = spec.ldpos;
    p.inv_freq = spec.inv_freq;
    p.heads = heads;
    p.dim = dim;
    p.pairs = spec.pairs;
    p.interleaved = spec.interleaved;
    if (spec.axis) memcpy(p.axis, spec.axis, static_cast<size_t>(spec.pairs));
    const int64_t want = static_cast<int64_t>(dev.sms) * 8;
    k_rope<<<static_cast<unsigned>(T < want ? T : want), kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace tq
