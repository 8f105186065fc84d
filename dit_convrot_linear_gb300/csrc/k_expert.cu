// A layer's experts around their products: the router's choice of k experts a
// token with its weights, the sort of the choices by expert, rows gathered by that
// order, and the weighted sum back into token order, with the gradients of the
// choice's weights and of the sum.
//
// All but the sort are bound by memory at many tokens and by a launch at few.

#include "tq_internal.cuh"

namespace tq {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ------------------------------------------------------------ the router

// Order of logits as unsigned numbers: 0 for -inf (never chosen), NaN above +inf (chosen
// first: the row's weights come out as NaN, not as a quiet choice).  The addition makes
// the two zeros one, and all NaN (a sum's is 0x7FFFFFFF).
constexpr uint32_t kLowest = 0x007FFFFFu;        // -inf, as the others before it is subtracted

__device__ __forceinline__ uint32_t logit_key(float x) {
    const int b = __float_as_int(x + 0.0f);
    return (static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u)) - kLowest;
}

__device__ __forceinline__ float key_logit(uint32_t key) {
    const uint32_t b = key + kLowest;
    return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

template <typename L>
__device__ __forceinline__ float load_logit(const L *p) {
    if constexpr (sizeof(L) == 4)
        return __ldg(p);
    else
        return bf16_bits_to_f32(__ldg(p));
}

// A warp a token; lane l holds experts l, l + 32, ...  The k-th largest of the lanes'
// largest keys is no larger than the k-th key: what reaches it is brought together in
// shared memory, a key a lane in the order of the experts (usually k to 2 k are), and
// each looks at the others for its place.  Where more than 32 reach it each choice looks
// through all keys.  Bound by the instructions: 16384
// tokens, 8 of 256 experts 10.1 us (13.9 with each lane's keys sorted instead); the
// logits' 17 MB take 2.5 at the copy rate.
template <typename L, int NI>
__global__ void __launch_bounds__(256) k_expert_topk(const L *__restrict__ X, int64_t T, int E, int64_t ld, int k,
                                                     int renorm, int32_t *__restrict__ ids,
                                                     float *__restrict__ weights) {
    __shared__ uint2 found_sh[8][32];
    const int lane = threadIdx.x & 31;
    uint2 *found = found_sh[threadIdx.x >> 5];
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < T; t += step) {
        const L *x = X + t * ld + lane;
        uint32_t key[NI], most = 0u;
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = lane + 32 * i < E ? logit_key(load_logit(x + 32 * i)) : 0u;
#pragma unroll
        for (int i = 0; i < NI; ++i) most = max(most, key[i]);
        // the softmax over all experts is relative to the largest logit
        const uint32_t top = __reduce_max_sync(kAll, most);
        float all = 0.0f;
        if (!renorm) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (key[i] != 0u) all += expf(key_logit(key[i]) - key_logit(top));
            all = warp_sum(all);
        }
        uint32_t mine = key[0];                  // one of those that may be chosen, of expert at
        int at = lane, many = 32;
        if constexpr (NI > 1) {
            many = 0;
            uint32_t bound = top;
            for (int n = 0; bound != 0u;) {
                n += __popc(__ballot_sync(kAll, most == bound));
                if (n >= k) break;
                if (most == bound) most = 0u;
                bound = __reduce_max_sync(kAll, most);
            }
            bound = max(bound, 1u);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const uint32_t b = __ballot_sync(kAll, key[i] >= bound);
                const int to = many + __popc(b & ((1u << lane) - 1u));
                if (key[i] >= bound && to < 32) found[to] = make_uint2(key[i], lane + 32 * i);
                many += __popc(b);
            }
            __syncwarp();
            const uint2 f = found[lane];
            mine = lane < many ? f.x : 0u;
            at = static_cast<int>(f.y);
            __syncwarp();                        // the next token's
        }
        int id = -1, rank = lane;                // this lane's choice, and which one it is
        uint32_t chosen = 0u;
        if (many <= 32) {
            // as many of them are larger, or equal and of a lower expert (the lanes that have
            // none keep their own places, which are behind)
            if (lane < many) rank = 0;
            for (int j = 0; j < many; ++j) {
                const uint32_t other = __shfl_sync(kAll, mine, j);
                if (lane < many && (other > mine || (other == mine && j < lane))) ++rank;
            }
            if (mine != 0u && rank < k) {
                chosen = mine;
                id = at;
            }
        } else {
            for (int j = 0; j < k; ++j) {
                uint32_t best = key[0];
                int e = lane;
#pragma unroll
                for (int i = 1; i < NI; ++i)
                    if (key[i] > best) {
                        best = key[i];
                        e = lane + 32 * i;
                    }
                const uint32_t win = __reduce_max_sync(kAll, best);
                if (win == 0u) break;
                e = static_cast<int>(__reduce_min_sync(kAll, best == win ? static_cast<uint32_t>(e) : 0xFFFFu));
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (lane + 32 * i == e) key[i] = 0u;
                if (lane == j) {
                    id = e;
                    chosen = win;
                }
            }
        }
        const float w = id >= 0 ? expf(key_logit(chosen) - key_logit(top)) : 0.0f;
        if (renorm) all = warp_sum(w);
        if (rank < k) {
            ids[t * k + rank] = id;
            weights[t * k + rank] = id >= 0 ? w / all : 0.0f;
        }
    }
}

// dlogits of the weights' gradients dw.  With the chosen ones' own softmax w:
//   w_i (dw_i - sum_j w_j dw_j) at the chosen, 0 elsewhere;
// with the softmax p over all experts: p_e (dw at e - sum_j p_j dw_j).
// 16384 tokens, 8 of 256 experts, fp32: 8.3 us (10.2 with a look at each choice for each
// logit in place of the trip through shared memory), 5.0 at the copy rate.
template <typename L, int NI>
__global__ void __launch_bounds__(256) k_expert_topk_grad(const L *__restrict__ X, int64_t T, int E, int64_t ld,
                                                          const int32_t *__restrict__ ids,
                                                          const float *__restrict__ dw, int k, int renorm,
                                                          L *__restrict__ dX, int64_t ldd, unsigned int *status) {
    __shared__ float at_sh[8][32 * NI];           // the chosen experts' part of dlogits, 0 at the others
    const int lane = threadIdx.x & 31;
    float *at = at_sh[threadIdx.x >> 5];
#pragma unroll
    for (int i = 0; i < NI; ++i) at[lane + 32 * i] = 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < T; t += step) {
        int id = -1;
        float d = 0.0f, v = 0.0f;
        if (lane < k) {
            id = ids[t * k + lane];
            if (id < -1 || id >= E) {
                atomicOr(status, kStatusIndex);
                id = -1;
            }
            if (id >= 0) {
                d = dw[t * k + lane];
                v = load_logit(X + t * ld + id);
            }
        }
        float x[NI];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            x[i] = !renorm && e < E ? load_logit(X + t * ld + e) : -INFINITY;
            top = x[i] > top || x[i] != x[i] ? x[i] : top;
        }
        if (renorm && id >= 0) top = v;
        bool nan = top != top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        if (__any_sync(kAll, nan)) top = __uint_as_float(0x7FC00000u);
        if (top == -INFINITY) top = 0.0f;
        float w = id >= 0 ? expf(v - top) : 0.0f;
        float total = w;
        if (!renorm) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) total += x[i] = lane + 32 * i < E ? expf(x[i] - top) : 0.0f;
        }
        total = warp_sum(total);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        w *= inv;
        const float mean = warp_sum(w * d);
        const float part = renorm ? w * (d - mean) : d;
        // (one that ids has twice gets both parts, in their order)
        const bool once = __match_any_sync(kAll, id) == 1u << lane;
        __syncwarp();
        if (__all_sync(kAll, once || id < 0)) {
            if (id >= 0) at[id] = part;
        } else {
            for (int j = 0; j < k; ++j) {
                if (lane == j && id >= 0) at[id] += part;
                __syncwarp();
            }
        }
        __syncwarp();
        float r[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) r[i] = at[lane + 32 * i];
        __syncwarp();
        if (id >= 0) at[id] = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e >= E) continue;
            if (!renorm) r[i] = x[i] * inv * (r[i] - mean);
            if constexpr (sizeof(L) == 4)
                dX[t * ldd + e] = r[i];
            else
                dX[t * ldd + e] = f32_to_bf16_bits(r[i]);
        }
    }
}

// ------------------------------------------------------------ the sort

// A counting sort by one cluster.  Each warp counts the experts of its own piece of the
// choices; the counts are summed over warps, CTAs (through distributed shared memory)
// and experts; then each warp places its piece.  Pieces are in order, and so are the
// choices within one, so equal experts stay in order.  131072 choices of 256 experts take
// 10.4 us, more than half of it in the placing: the instructions of a warp's eight steps,
// 32 warps an SM (10.7 with indexes of 64 bits).  Before that: eight CTAs 16.4, one 102; a
// second kernel that scatters the tokens from all SMs 12.2; the tokens put in order in
// shared memory first 10.9; a match among the lanes in place of a vote for each bit 15.8,
// masks in shared memory 11.0.  Few choices go to one CTA: 2048 take 5.0 by it and 5.5 by
// the cluster, 4096 6.3 and 5.7.
constexpr int kSortWarps = 32, kSortCtas = 16, kSortAhead = 8;
constexpr int64_t kSortOneCta = 2048;            // choices that one CTA sorts alone

__device__ __forceinline__ int remote_int(uint32_t addr, int cta) {
    uint32_t at;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(cta));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// (.aligned: a warp's lanes have to come together, also after a loop that they leave at
// different times)
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int BITS>
__global__ void __launch_bounds__(32 * kSortWarps) k_expert_sort(const int32_t *__restrict__ ids, uint32_t n, uint32_t k,
                                                                 int E, int32_t *__restrict__ offsets,
                                                                 int32_t *__restrict__ token,
                                                                 int32_t *__restrict__ place, unsigned int *status) {
    extern __shared__ int cnt[];                 // [warps][E] counts, then [E] this CTA's, then [E] bases
    int *sum_cta = cnt + kSortWarps * E, *base = sum_cta + E;
    __shared__ int part[kSortWarps + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ctas = gridDim.x, cta = blockIdx.x;
    for (int i = threadIdx.x; i < kSortWarps * E; i += blockDim.x) cnt[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    // (n < 2^31, and all of it in 32 bits: the instructions count)
    const uint32_t warps = ctas * kSortWarps, per = ((n + warps - 1) / warps + 31) / 32 * 32;
    const uint32_t f0 = min((cta * kSortWarps + warp) * per, n), f1 = min(f0 + per, n);
    int *mine = cnt + warp * E;
    // f(position, expert or -1, the number given) for the piece's choices in order
    auto walk = [&](auto &&f) {
        for (uint32_t at = f0; at < f1; at += 32 * kSortAhead) {
            int e[kSortAhead];
#pragma unroll
            for (int i = 0; i < kSortAhead; ++i) {
                const uint32_t g = at + 32 * i + lane;
                e[i] = g < f1 ? __ldg(ids + g) : -1;
            }
#pragma unroll
            for (int i = 0; i < kSortAhead; ++i) {
                if (at + 32 * i >= f1) break;
                const int v = static_cast<unsigned>(e[i]) < static_cast<unsigned>(E) ? e[i] : -1;
                f(at + 32 * i + lane, v, e[i]);
            }
        }
    };
    __syncthreads();
    walk([&](uint32_t, int e, int given) {
        if (given != e) atomicOr(status, kStatusIndex);
        if (e >= 0) atomicAdd(mine + e, 1);
    });
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = sum;
            sum += c;
        }
        sum_cta[e] = sum;
    }
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // a thread an expert (E <= 1024): choices of it in all CTAs, and in those before this one
    const int e = threadIdx.x;
    int all = 0, before = 0;
    if (e < E) {
        if (ctas > 1) {
            const uint32_t addr = static_cast<uint32_t>(__cvta_generic_to_shared(sum_cta + e));
#pragma unroll
            for (int c = 0; c < kSortCtas; ++c) {
                const int v = remote_int(addr, c);
                all += v;
                before += c < cta ? v : 0;
            }
        } else {
            all = sum_cta[e];
        }
    }
    if (ctas > 1) cluster_arrive();              // the other CTAs' counts have been read
    int s = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, s, o);
        if (lane >= o) s += v;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int v = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += u;
        }
        part[lane] = v;
    }
    __syncthreads();
    const int start = s - all + (warp > 0 ? part[warp - 1] : 0), total = part[kSortWarps - 1];
    if (e < E) {
        base[e] = start + before;
        if (cta == 0) offsets[e] = start;
    }
    if (cta == 0 && threadIdx.x == 0) offsets[E] = total;
    __syncthreads();
    // the choice's token: its number by k, a step of 32 at a time
    const uint32_t by = 32 / k, over = 32 % k;
    uint32_t tok = (f0 + lane) / k, rest = f0 + lane - tok * k;
    walk([&](uint32_t f, int e, int) {
        // the lanes with the same expert: a vote for each bit of its number
        uint32_t same = __ballot_sync(kAll, e >= 0);
#pragma unroll
        for (int b = 0; b < BITS; ++b) {
            const bool one = (e >> b) & 1;
            const uint32_t v = __ballot_sync(kAll, one);
            same &= one ? v : ~v;
        }
        int at = -1;
        if (e >= 0) {
            at = base[e] + mine[e] + __popc(same & ((1u << lane) - 1u));
            token[at] = static_cast<int32_t>(tok);
        }
        if (f < f1) place[f] = at;
        tok += by;
        rest += over;
        if (rest >= k) {
            rest -= k;
            ++tok;
        }
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    });
    for (uint32_t i = total + cta * blockDim.x + threadIdx.x; i < n; i += ctas * blockDim.x) token[i] = -1;
    if (ctas > 1) cluster_wait();                // nobody leaves while its counts may still be read
}

// ------------------------------------------------------------ rows there and back

// 16 bytes of a row as fp32 values
template <typename V>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(const uint4 &u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Piece<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = f32_to_bf16_bits(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// A warp a row, or a quarter of one: four 16-byte pieces a lane on their way at once.
// Bound by the stores: 65536 rows of 4096 bf16 out of 8192, an eighth left out, 126 us
// (470 MB written at 3.7 TB/s; 124 with a thread a piece); with none left out 137 (3.9 TB/s),
// and zeros filled in over the same 537 MB, with nothing read, take 134 (4.0 TB/s); 8192
// out of 4096 13.3 to 17 (15.9).
__global__ void __launch_bounds__(256) k_expert_gather(const uint4 *__restrict__ X, int64_t rows_x, int pieces,
                                                       int parts, int64_t ldx, const int32_t *__restrict__ rows,
                                                       int64_t M, uint4 *__restrict__ Y, int64_t ldy,
                                                       unsigned int *status) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8, n = M * parts;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < n; i += step) {
        const int64_t m = i / parts;
        const int part = static_cast<int>(i - m * parts);
        const int32_t r = __ldg(rows + m);
        if (r < 0 || r >= rows_x) {
            if (r != -1 && lane == 0) atomicOr(status, kStatusIndex);
            continue;
        }
        const uint4 *x = X + r * ldx;
        uint4 *y = Y + m * ldy;
        for (int c0 = 128 * part + lane; c0 < pieces; c0 += 128 * parts) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c0 + 32 * u < pieces) v[u] = __ldg(x + c0 + 32 * u);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c0 + 32 * u < pieces) y[c0 + 32 * u] = v[u];
        }
    }
}

constexpr int kGradRows = 4;            // of the gradients

// A thread a 16-byte piece of a token's row: the sum over its choices in their
// order, in fp32, R rows on their way at once.  Eight choices of 8192 tokens, an eighth
// of them none, 4096 wide, bf16: 84 us, 6390 GB/s, with R = 4; 106 with 8, which leaves
// room for three CTAs an SM.  Two choices of 4096 tokens: 17.8 with R = 2 (35.7 with 8).
template <typename V, int R>
__global__ void __launch_bounds__(256) k_expert_combine(const uint4 *__restrict__ Y, int64_t rows, int pieces,
                                                        int64_t ldy, const int32_t *__restrict__ place,
                                                        const float *__restrict__ weights, int64_t T, int k,
                                                        uint4 *__restrict__ O, int64_t ldo, unsigned int *status) {
    using P = Piece<V>;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, on = step / pieces;
    const int over = static_cast<int>(step - on * pieces);
    int64_t t = i / pieces;
    int c = static_cast<int>(i - t * pieces);
    for (; t < T; t += on, c += over) {
        if (c >= pieces) {
            c -= pieces;
            if (++t >= T) break;
        }
        float sum[P::N] = {};
        for (int j0 = 0; j0 < k; j0 += R) {
            uint4 row[R];
            float w[R];
            bool in[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int32_t at = j0 + j < k ? __ldg(place + t * k + j0 + j) : -1;
                in[j] = at >= 0 && at < rows;
                if (!in[j] && at != -1 && c == 0) atomicOr(status, kStatusIndex);
                w[j] = weights && j0 + j < k ? __ldg(weights + t * k + j0 + j) : 1.0f;
                if (in[j]) row[j] = ldg_stream(Y + at * ldy + c);
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (!in[j]) continue;
                float v[P::N];
                P::widen(row[j], v);
#pragma unroll
                for (int q = 0; q < P::N; ++q) sum[q] = fmaf(w[j], v[q], sum[q]);
            }
        }
        O[t * ldo + c] = P::narrow(sum);
    }
}

// A CTA a token: dY of each of its rows, w * dO, and dw = dO . Y, kGradRows rows on
// their way at once.  Eight choices of 4096 tokens, 4096 wide, bf16: 90 us, 6310 GB/s,
// with the registers of four CTAs an SM (100 with three; two rows at once 107).
constexpr int kGradThreads = 256;
template <typename V>
__global__ void __launch_bounds__(kGradThreads, 4) k_expert_combine_grad(
    const uint4 *__restrict__ dO, int64_t ldo, const uint4 *__restrict__ Y, int64_t rows, int pieces, int64_t ldy,
    const int32_t *__restrict__ place, const float *__restrict__ weights, int64_t T, int k, uint4 *__restrict__ dY,
    int64_t lddy, float *__restrict__ dw, unsigned int *status) {
    using P = Piece<V>;
    __shared__ float part[kGradRows][kGradThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        for (int j0 = 0; j0 < k; j0 += kGradRows) {
            int32_t at[kGradRows];
            float w[kGradRows], dot[kGradRows];
#pragma unroll
            for (int j = 0; j < kGradRows; ++j) {
                at[j] = j0 + j < k ? __ldg(place + t * k + j0 + j) : -1;
                w[j] = weights && j0 + j < k ? __ldg(weights + t * k + j0 + j) : 1.0f;
                dot[j] = 0.0f;
                if (at[j] < -1 || at[j] >= rows) {
                    if (threadIdx.x == 0) atomicOr(status, kStatusIndex);
                    at[j] = -1;
                }
            }
            for (int c = threadIdx.x; c < pieces; c += kGradThreads) {
                uint4 row[kGradRows];
                if (dw)
#pragma unroll
                    for (int j = 0; j < kGradRows; ++j)
                        if (at[j] >= 0) row[j] = ldg_stream(Y + at[j] * ldy + c);
                float d[P::N];
                P::widen(__ldg(dO + t * ldo + c), d);
#pragma unroll
                for (int j = 0; j < kGradRows; ++j) {
                    if (at[j] < 0) continue;
                    float v[P::N];
                    if (dw) {
                        P::widen(row[j], v);
#pragma unroll
                        for (int q = 0; q < P::N; ++q) dot[j] = fmaf(d[q], v[q], dot[j]);
                    }
#pragma unroll
                    for (int q = 0; q < P::N; ++q) v[q] = d[q] * w[j];
                    dY[at[j] * lddy + c] = P::narrow(v);
                }
            }
            if (dw) {
#pragma unroll
                for (int j = 0; j < kGradRows; ++j) {
                    dot[j] = warp_sum(dot[j]);
                    if ((threadIdx.x & 31) == 0) part[j][threadIdx.x >> 5] = dot[j];
                }
                __syncthreads();
                if (threadIdx.x < kGradRows && j0 + threadIdx.x < k) {
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < kGradThreads / 32; ++i) s += part[threadIdx.x][i];
                    dw[t * k + j0 + threadIdx.x] = s;
                }
                __syncthreads();
            }
        }
    }
}

unsigned grid_of(int64_t ctas, const DeviceInfo &dev, int each) {
    const int64_t most = static_cast<int64_t>(dev.sms) * each;
    return static_cast<unsigned>(ctas < most ? ctas : most);
}

// F<NI> for the 32-expert pieces of E
template <template <int> class F, typename... A>
tq_status by_experts(int64_t E, A... a) {
    if (E <= 32) return F<1>::run(a...);
    if (E <= 64) return F<2>::run(a...);
    if (E <= 128) return F<4>::run(a...);
    if (E <= 256) return F<8>::run(a...);
    if (E <= 512) return F<16>::run(a...);
    return F<32>::run(a...);
}

}  // namespace

namespace {
template <int NI>
struct Topk {
    static tq_status run(const void *x, int type, int64_t T, int E, int64_t ld, int k, int renorm, int32_t *ids, float *w,
                         unsigned grid, cudaStream_t s) {
        if (type == 0)
            return launch_pdl(k_expert_topk<float, NI>, grid, 256, s, static_cast<const float *>(x), T, E, ld, k, renorm,
                              ids, w);
        return launch_pdl(k_expert_topk<uint16_t, NI>, grid, 256, s, static_cast<const uint16_t *>(x), T, E, ld, k,
                          renorm, ids, w);
    }
};
template <int NI>
struct TopkGrad {
    static tq_status run(const void *x, int type, int64_t T, int E, int64_t ld, const int32_t *ids, const float *dw,
                         int k, int renorm, void *dx, int64_t ldd, unsigned int *status, unsigned grid, cudaStream_t s) {
        if (type == 0)
            return launch_pdl(k_expert_topk_grad<float, NI>, grid, 256, s, static_cast<const float *>(x), T, E, ld, ids,
                              dw, k, renorm, static_cast<float *>(dx), ldd, status);
        return launch_pdl(k_expert_topk_grad<uint16_t, NI>, grid, 256, s, static_cast<const uint16_t *>(x), T, E, ld,
                          ids, dw, k, renorm, static_cast<uint16_t *>(dx), ldd, status);
    }
};
}  // namespace

tq_status launch_expert_topk(const void *logits, int type, int64_t T, int64_t E, int64_t ld, int k, int renorm,
                             int32_t *ids, float *weights, const DeviceInfo &dev, cudaStream_t s) {
    return by_experts<Topk>(E, logits, type, T, static_cast<int>(E), ld, k, renorm, ids, weights,
                            grid_of((T + 7) / 8, dev, 64), s);
}

tq_status launch_expert_topk_grad(const void *logits, int type, int64_t T, int64_t E, int64_t ld, const int32_t *ids,
                                  const float *dw, int k, int renorm, void *dlogits, int64_t ldd,
                                  const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    return by_experts<TopkGrad>(E, logits, type, T, static_cast<int>(E), ld, ids, dw, k, renorm, dlogits, ldd, status,
                                grid_of((T + 7) / 8, dev, 64), s);
}

tq_status launch_expert_sort(const int32_t *ids, int64_t T, int k, int64_t E, int32_t *offsets, int32_t *token,
                             int32_t *place, const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status || dev.id < 0 || dev.id >= 64) return TQ_ERR_DEVICE;
    const int bytes = static_cast<int>((kSortWarps * E + 2 * E) * 4);
    auto kern = E <= 64 ? k_expert_sort<6> : (E <= 256 ? k_expert_sort<8> : k_expert_sort<10>);
    static bool configured[64] = {false};
    if (!configured[dev.id]) {
        for (auto f : {k_expert_sort<6>, k_expert_sort<8>, k_expert_sort<10>}) {
            cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (kSortWarps + 2) * TQ_MAX_EXPERTS * 4);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return cuda_fail(e);
        }
        configured[dev.id] = true;
    }
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    const unsigned ctas = T * k <= kSortOneCta ? 1u : static_cast<unsigned>(kSortCtas);
    attr[0].val.clusterDim = {ctas, 1u, 1u};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * kSortWarps);
    cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, ids, static_cast<uint32_t>(T * k),
                                             static_cast<uint32_t>(k), static_cast<int>(E), offsets, token,
                                             place, status);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

tq_status launch_expert_gather(const void *X, int type, int64_t rows_x, int64_t W, int64_t ldx, const int32_t *rows,
                               int64_t M, void *Y, int64_t ldy, const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    const int each = type == 0 ? 4 : 8;          // values of 16 bytes
    const int pieces = static_cast<int>(W / each), parts = pieces > 384 ? 4 : (pieces + 127) / 128;
    return launch_pdl(k_expert_gather, grid_of((M * parts + 7) / 8, dev, 8), 256, s, static_cast<const uint4 *>(X), rows_x,
                      pieces, parts, ldx / each, rows, M, static_cast<uint4 *>(Y), ldy / each, status);
}

tq_status launch_expert_combine(const void *Y, int type, int64_t rows, int64_t W, int64_t ldy, const int32_t *place,
                                const float *weights, int64_t T, int k, void *O, int64_t ldo, const DeviceInfo &dev,
                                cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    const int each = type == 0 ? 4 : 8, pieces = static_cast<int>(W / each);
    const unsigned grid = grid_of((T * pieces + 255) / 256, dev, 8);
    auto y = static_cast<const uint4 *>(Y);
    auto o = static_cast<uint4 *>(O);
    auto kern = k <= 2 ? (type == 0 ? k_expert_combine<float, 2> : k_expert_combine<uint16_t, 2>)
                       : (type == 0 ? k_expert_combine<float, 4> : k_expert_combine<uint16_t, 4>);
    return launch_pdl(kern, grid, 256, s, y, rows, pieces, ldy / each, place, weights, T, k, o, ldo / each, status);
}

tq_status launch_expert_combine_grad(const void *dO, int64_t ldo, const void *Y, int type, int64_t rows, int64_t W,
                                     int64_t ldy, const int32_t *place, const float *weights, int64_t T, int k,
                                     void *dY, int64_t lddy, float *dw, const DeviceInfo &dev, cudaStream_t s) {
    unsigned int *status = status_word();
    if (!status) return TQ_ERR_DEVICE;
    const int each = type == 0 ? 4 : 8, pieces = static_cast<int>(W / each);
    const unsigned grid = grid_of(T, dev, 8);
    auto d = static_cast<const uint4 *>(dO);
    auto y = static_cast<const uint4 *>(Y);
    auto o = static_cast<uint4 *>(dY);
    return launch_pdl(type == 0 ? k_expert_combine_grad<float> : k_expert_combine_grad<uint16_t>, grid, kGradThreads, s,
                      d, ldo / each, y, rows, pieces, ldy / each, place, weights, T, k, o, lddy / each, dw, status);
}

}  // namespace tq
