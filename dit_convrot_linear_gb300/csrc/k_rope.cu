// Rotary positions with one or more axes (Su et al., "RoFormer", 2021): pair p
// of every head of token t turns by the angle pos[axis(p)][t] * inv_freq[p].
//
// Bound by memory: 2 B read and 2 B written per value.  A CTA takes a few
// tokens at a time: it forms their sines and cosines once (a thread a pair, the
// angle in fp64), then turns all their heads, eight pairs a thread as two
// 16-byte pieces half a head apart, or four neighbouring pairs as one.  8190
// tokens of 48 heads of 128 on three axes: 41 us, 73 % of the copy rate (30 us for
// the bytes; a CTA's rows are loaded after its angles, and those take fp64, for
// which this GPU has few lanes); 32 tokens of 40 heads 2.7 us, a launch's own time.

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
    int batch;                               // tokens a CTA takes at a time
    uint8_t axis[TQ_ROPE_MAX_DIM / 2];
};

constexpr int kTurns = 512;                  // sines and cosines a CTA holds

// cos and sin of pos * f.  The product of an int32 and an fp32 number is exact
// in fp64 (31 + 24 bits, rounded once to 53), and one multiple of 2 pi (in two
// parts) taken off it in fp64 leaves an argument within [-pi, pi] whose error
// stays below 2^-20 for every int32 position and |f| <= 1.
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

__device__ __forceinline__ void turn(float &a, float &b, const float2 &w) {
    const float x = a * w.x - b * w.y;
    b = b * w.x + a * w.y;
    a = x;
}

__device__ __forceinline__ void widen(const uint4 &u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// KIND 0: pairs of values p and p + pairs, pairs a multiple of 8; 1:
// neighbouring values, pairs a multiple of 4; 2: any, a pair a thread.
template <int KIND>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[kTurns];
    pdl_launch_dependents();
    pdl_wait();
    const int rest = p.dim - 2 * p.pairs;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.batch; t0 < p.T;
         t0 += static_cast<int64_t>(gridDim.x) * p.batch) {
        const int nt = p.T - t0 < p.batch ? static_cast<int>(p.T - t0) : p.batch;
        __syncthreads();
        for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
            const int t = i / p.pairs, q = i - t * p.pairs;
            cs[i] = turn_of(__ldg(p.pos + p.axis[q] * p.ldpos + t0 + t), __ldg(p.inv_freq + q));
        }
        __syncthreads();
        // work items: (token, head, piece), pieces fastest
        const int per_head = KIND == 0 ? p.pairs / 8 : KIND == 1 ? p.pairs / 4 : p.pairs;
        const int per_token = per_head * p.heads;
        for (int i = threadIdx.x; i < nt * per_token; i += kThreads) {
            const int t = i / per_token, k = i - t * per_token;
            const int h = k / per_head, c = k - h * per_head;
            const uint16_t *x = p.X + (t0 + t) * p.ldx + h * p.dim;
            uint16_t *y = p.Y + (t0 + t) * p.ldy + h * p.dim;
            const float2 *w = cs + t * p.pairs;
            if constexpr (KIND == 0) {
                float a[8], b[8];
                const uint4 ua = *reinterpret_cast<const uint4 *>(x + 8 * c);
                const uint4 ub = *reinterpret_cast<const uint4 *>(x + p.pairs + 8 * c);
                widen(ua, a);
                widen(ub, b);
#pragma unroll
                for (int e = 0; e < 8; ++e) turn(a[e], b[e], w[8 * c + e]);
                *reinterpret_cast<uint4 *>(y + 8 * c) = narrow(a);
                *reinterpret_cast<uint4 *>(y + p.pairs + 8 * c) = narrow(b);
            } else if constexpr (KIND == 1) {
                float a[8];
                widen(*reinterpret_cast<const uint4 *>(x + 8 * c), a);
#pragma unroll
                for (int e = 0; e < 4; ++e) turn(a[2 * e], a[2 * e + 1], w[4 * c + e]);
                *reinterpret_cast<uint4 *>(y + 8 * c) = narrow(a);
            } else {
                const int step = p.interleaved ? 1 : p.pairs, at = p.interleaved ? 2 * c : c;
                float a = bf16_bits_to_f32(x[at]), b = bf16_bits_to_f32(x[at + step]);
                turn(a, b, w[c]);
                y[at] = f32_to_bf16_bits(a);
                y[at + step] = f32_to_bf16_bits(b);
            }
        }
        if (rest == 0 || p.X == p.Y) continue;
        // the values past the pairs
        for (int i = threadIdx.x; i < nt * p.heads * rest; i += kThreads) {
            const int t = i / (p.heads * rest), k = i - t * p.heads * rest;
            const int h = k / rest, at = h * p.dim + 2 * p.pairs + (k - h * rest);
            p.Y[(t0 + t) * p.ldy + at] = p.X[(t0 + t) * p.ldx + at];
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
    const int kind = p.interleaved ? (p.pairs % 4 == 0 ? 1 : 2) : (p.pairs % 8 == 0 ? 0 : 2);
    // tokens at a time: as many turns as fit, but no fewer CTAs than fill the GPU
    const int64_t most = static_cast<int64_t>(dev.sms) * 8;
    int64_t batch = kTurns / p.pairs;
    if (batch > (T + most - 1) / most) batch = (T + most - 1) / most;
    p.batch = static_cast<int>(batch < 1 ? 1 : batch);
    const int64_t blocks = (T + p.batch - 1) / p.batch;
    auto kern = kind == 0 ? k_rope<0> : kind == 1 ? k_rope<1> : k_rope<2>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace tq
