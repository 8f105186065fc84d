// Attention over the 4-bit cache, one CTA per query row and head.
//
// o = H^T softmax(scale (H q) . k') v' with k' = s_k (u - 8), v' = s_v (u - 8):
// one pass over the row's positions in steps of 128, a running maximum and sum
// in fp32, a thread per position for the scores and per value column for the
// weighted sum.

#include <math_constants.h>

#include "tq_kv4.cuh"

namespace tq {
namespace {

constexpr int kStep = 128;

template <int E>
__global__ void __launch_bounds__(kStep)
k_kv4_attn_rows(const __grid_constant__ tq_kv4 kv, const __grid_constant__ Kv4Attn a, unsigned int *status) {
    constexpr int D = 32 * E;
    constexpr int C = (D + kStep - 1) / kStep;       // value columns a thread
    __shared__ float q_sh[D], o_sh[D], w_sh[kStep], red[2][kStep / 32];
    __shared__ const unsigned char *blk_sh[kStep / kKvBlock];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hq = blockIdx.x % a.heads_q;
    const int64_t t = blockIdx.x / a.heads_q;
    const int h = hq / (a.heads_q / kv.heads);
    bool bad = false;

    // the sequence that owns this row
    int64_t b = -1;
    KvSeq q = {0, 0, 0};
    for (int64_t i = 0; i < kv.nseq; ++i) {
        const KvSeq c = kv_seq(kv, i, bad);
        if (t >= c.start && t < static_cast<int64_t>(c.start) + c.n) {
            b = i;
            q = c;
        }
    }
    if (bad && tid == 0) atomicOr(status, kStatusIndex);
    if (b < 0) return;
    const int64_t pos = q.len - q.n + (t - q.start);
    const int64_t hi = pos < 0 ? 0 : a.causal && pos + 1 < q.len ? pos + 1 : q.len;
    const int64_t lo = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;

    if (warp == 0) {
        float v[8];
        load_bf16<E, float>(a.Q + t * a.ldq + static_cast<int64_t>(hq) * D + lane * E, v);
        warp_fwht<E, float>(v);
        const float c = sqrtf(1.0f / D);
#pragma unroll
        for (int e = 0; e < E; ++e) q_sh[lane * E + e] = c * v[e];
    }
    float m = -CUDART_INF_F, l = 0.0f, acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.0f;
    for (int64_t base = lo / kKvBlock * kKvBlock; base < hi; base += kStep) {
        __syncthreads();
        if (tid < kStep / kKvBlock) {
            const int64_t at = base + tid * kKvBlock;
            const int page = at < hi ? kv_page(kv, b, static_cast<int>(at)) : -1;
            blk_sh[tid] = page >= 0 ? kv_block(kv, page, h, static_cast<int>(at % kv.page_size)) : nullptr;
            if (at < hi && page < 0) atomicOr(status, kStatusIndex);
        }
        __syncthreads();
        const int64_t j = base + tid;
        const unsigned char *blk = blk_sh[tid / kKvBlock];
        const int r = tid % kKvBlock;
        const bool see = blk && j >= lo && j < hi;
        float x = -CUDART_INF_F;
        if (see) {
            float sum = 0.0f;
            for (int i = 0; i < D / 2; ++i) {
                const int u = blk[r * (D / 2) + i];
                sum = fmaf(q_sh[2 * i], static_cast<float>((u & 15) - 8), sum);
                sum = fmaf(q_sh[2 * i + 1], static_cast<float>((u >> 4) - 8), sum);
            }
            x = sum * reinterpret_cast<const float *>(blk + 16 * D)[r] * a.scale;
        }
        float mx = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) red[0][warp] = mx;
        __syncthreads();
        mx = m;
#pragma unroll
        for (int w = 0; w < kStep / 32; ++w) mx = fmaxf(mx, red[0][w]);
        const float base_m = mx > -CUDART_INF_F ? mx : 0.0f;
        const float w = see ? expf(x - base_m) : 0.0f;
        const float fix = expf(m - base_m);
        w_sh[tid] = see ? w * reinterpret_cast<const float *>(blk + 16 * D)[16 + r] : 0.0f;
        float sum = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) red[1][warp] = sum;
        __syncthreads();
        l *= fix;
#pragma unroll
        for (int k = 0; k < kStep / 32; ++k) l += red[1][k];
        m = mx;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int d = tid + c * kStep;
            acc[c] *= fix;
            if (d >= D) continue;
            for (int k = 0; k < kStep; ++k) {
                const unsigned char *vb = blk_sh[k / kKvBlock];
                if (!vb) continue;
                const int row = k % kKvBlock;
                const int u = vb[8 * D + (row >> 1) * D + (d >> 2) * 4 + (row & 1) * 2 + ((d & 3) >> 1)];
                acc[c] = fmaf(w_sh[k], static_cast<float>(((u >> (4 * (d & 1))) & 15) - 8), acc[c]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (tid + c * kStep < D) o_sh[tid + c * kStep] = l > 0.0f ? acc[c] / l : 0.0f;
    __syncthreads();
    if (warp == 0) {
        float v[8];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = o_sh[lane * E + e];
        warp_fwht<E, float>(v);
        const float c = sqrtf(1.0f / D);
        uint16_t *o = a.O + t * a.ldo + static_cast<int64_t>(hq) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = f32_to_bf16_bits(c * v[e]);
        if (a.lse && lane == 0) a.lse[t * a.heads_q + hq] = l > 0.0f ? m + logf(l) : -CUDART_INF_F;
    }
}

}  // namespace

size_t kv4_workspace_bytes(const DeviceInfo &dev) {
    (void)dev;
    return 256;
}

tq_status launch_kv4_attention(const tq_kv4 &kv, const Kv4Attn &a, const DeviceInfo &dev, cudaStream_t s) {
    (void)dev;
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    auto kern = kv.dim == 64 ? k_kv4_attn_rows<2> : kv.dim == 128 ? k_kv4_attn_rows<4> : k_kv4_attn_rows<8>;
    kern<<<static_cast<unsigned>(kv.tokens * a.heads_q), kStep, 0, s>>>(kv, a, status);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace tq
