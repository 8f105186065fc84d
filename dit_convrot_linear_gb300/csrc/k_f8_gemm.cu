// The product of 8-bit floating-point operands with a scale for each block of 128,
//   Y[m][n] = sum_b sx[b][m] * sw[n / 128][b] * sum_{k in block b} xq[m][k] * wq[n][k],
// of one matrix, or of one matrix an expert over rows sorted by expert, on tcgen05
// (kind::f8f6f4: e4m3 operands as they are, at twice the rate of fp16).
//
// A pair of CTAs (tcgen05 cta_group::2) computes 256 output columns (weight rows,
// 128 a CTA: one scale block) of up to NT tokens.  The weights are the MMA's M side
// and the tokens its N side, so that the tile follows the number of tokens in steps
// of 16: an expert's few rows cost no empty rows of a 128-row tile.  A step of K is
// one scale block, four MMAs of 32; the accumulator of each step lies in TMEM of its
// own and the drain warps add it, times its scales, to the sums in their registers:
//   acc += (sx[b][token] * sw[block][b]) * part.
// Per CTA:
//   drain warps  (a TMEM lane quarter each; with NT = 256 two a quarter, half the
//                tokens each) multiply and add, and write Y;
//   MMA warp     allocates TMEM for the pair; in the even CTA one thread issues;
//   copy warp    tensor copies of both operands into the ring (128-byte swizzle);
//   scale warp   the tokens' scales of each step into a ring of their own.
//
// The work is a list of tiles (expert, 256 columns, up to NT tokens).  Whole rounds
// of tiles go to the pairs one by one; the K steps of a last round that would leave
// pairs idle are shared out evenly.  A pair that has only part of a tile's steps
// stores its sums, and the warp that comes last at the tile's counter adds all
// parts in the order of K: nobody waits, and the order does not depend on time.
// Every wait on an mbarrier is bounded: on expiry the CTA records it in the status
// word, stops, lets what is in flight finish (bounded), frees its TMEM and returns.

#include "tq_tc.cuh"

namespace tq {
namespace {

constexpr int kRowsW = 128;               // weight rows a CTA
constexpr int kStepK = 128;               // K of a step: one scale block
constexpr int kWBytes = kRowsW * kStepK;  // a stage's weights
constexpr int kBoxRows = 32;              // token rows of one tensor copy
constexpr long long kF8WaitLimit = 4000000000ll;   // clock cycles, about 2 s
constexpr unsigned int kStatusF8Timeout = 64u;

// NT tokens a tile.  256: as many as an MMA takes.  64: for few tokens, where the
// weights' stream is all there is: ten stages of weights in flight.
template <int NT_>
struct F8Plan {
    static constexpr int NT = NT_;
    static constexpr bool WIDE = NT == 256;
    static constexpr int DRAIN = WIDE ? 8 : 4;                 // drain warps
    static constexpr int THREADS = (DRAIN + 4) * 32;
    static constexpr int COLS = NT / (DRAIN / 4);              // tokens a drain warp
    static constexpr int STAGES = WIDE ? 6 : 10;
    static constexpr int X_BYTES = NT / 2 * kStepK;
    static constexpr int STAGE = kWBytes + X_BYTES;
    static constexpr int ACCS = WIDE ? 2 : 4;                  // accumulators in TMEM
    static constexpr int TMEM = NT * ACCS;
    static constexpr int SCALES = WIDE ? 6 : 12;               // slots of the scale ring
    static constexpr int OUT_ROWS = 16;                        // tokens a warp turns at once
    static constexpr int OUT_PITCH = 80;                       // bytes: 32 bf16 columns and padding
    static constexpr int OFF_SCALES = STAGES * STAGE;
    static constexpr int OFF_OUT = OFF_SCALES + SCALES * NT * 4;
    static constexpr int OFF_BARS = OFF_OUT + DRAIN * OUT_ROWS * OUT_PITCH;
    static constexpr int NBARS = 2 * STAGES + 2 * ACCS + 2 * SCALES + 1;
    static constexpr int OFF_LIST = OFF_BARS + (NBARS * 8 + 15) / 16 * 16;
    // the list of experts: rows before, tiles before (E + 1 numbers each)
    static constexpr int smem(int64_t experts) { return OFF_LIST + static_cast<int>(experts + 1) * 12 + 16; }
    static constexpr int SLOT = DRAIN * 32 * (COLS / 2) * 8;   // bytes of a CTA's partial tile
};
static_assert(F8Plan<256>::smem(TQ_MAX_EXPERTS) <= 227 * 1024 && F8Plan<64>::smem(TQ_MAX_EXPERTS) <= 227 * 1024,
              "shared memory");

constexpr int kF8MaxDrain = 8;

struct F8Params {
    const float *sx;
    int64_t M;
    const int32_t *offsets;
    int experts;
    const float *sw;
    int N, ksteps, nblocks, ntiles;      // nblocks: scale blocks of N; ntiles: 256-column tiles
    void *Y;
    int64_t ldy;
    int ytype, vec;                      // vec: rows of Y are 16-byte aligned
    unsigned int *status;
    unsigned int *counters;              // [pairs][2 CTAs][kF8MaxDrain]
    unsigned char *slots;                // [pairs][2][2 CTAs][SLOT]
    int min_steps;                       // K steps a pair takes of split tiles, at least
};

// A piece of work: the tile's place, K steps k0 .. k1 - 1, and for a piece of a
// split tile the pairs that have its first and last step.
struct F8Seg {
    int e, ntile, m0, cols, k0, k1;      // cols: tokens of the tile (at most NT)
    int mma_n;                           // cols rounded up to 16
    bool whole;
    int first, last;
};

struct F8List {
    const int *row0, *rows, *tiles;      // in shared memory: an expert's first row, rows, tiles before it
    int experts, total;                  // total: token tiles of all experts
};

template <int NT>
struct F8Iter {
    const F8List &l;
    int pair, pairs, ksteps, ntiles, whole_tiles, i, use, first_pair;
    long long units, u0, u;
    __device__ F8Iter(const F8List &list, const F8Params &p, int pair_, int pairs_)
        : l(list), pair(pair_), pairs(pairs_), ksteps(p.ksteps), ntiles(p.ntiles), i(0) {
        const int tiles = l.total * ntiles;
        const int rest = tiles % pairs;
        // the last round is split where it would leave a good part of the pairs idle
        const bool split = rest > 0 && rest * 100 < pairs * 85;
        whole_tiles = split ? tiles - rest : tiles;
        units = split ? static_cast<long long>(rest) * ksteps : 0;
        use = pairs;                     // pairs that share the split steps
        if (units < static_cast<long long>(pairs) * p.min_steps)
            use = max(1, static_cast<int>(units / p.min_steps));
        u0 = pair < use ? units * pair / use : 0;
        u = pair < use ? units * (pair + 1) / use : 0;
    }
    __device__ int owner(long long x) const {      // the pair whose steps include x
        int q = static_cast<int>(x * use / units);
        while (q + 1 < use && units * (q + 1) / use <= x) ++q;
        while (q > 0 && units * q / use > x) --q;
        return q;
    }
    __device__ void place(int tile, F8Seg &s) const {
        int lo = 0, hi = l.experts;      // tiles[lo] <= tile / ntiles < tiles[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (static_cast<long long>(l.tiles[mid]) * ntiles <= tile) lo = mid; else hi = mid;
        }
        const int at = tile - l.tiles[lo] * ntiles, parts = l.tiles[lo + 1] - l.tiles[lo];
        const int rows = l.rows[lo], each = ((rows + parts - 1) / parts + 15) / 16 * 16;
        const int part = at % parts;
        s.e = lo;
        s.ntile = at / parts;
        s.m0 = l.row0[lo] + part * each;
        s.cols = min(each, rows - part * each);
        s.mma_n = (max(s.cols, 1) + 15) / 16 * 16;
    }
    __device__ bool next(F8Seg &s) {
        const long long t = pair + static_cast<long long>(i) * pairs;
        if (t < whole_tiles) {
            ++i;
            place(static_cast<int>(t), s);
            s.k0 = 0;
            s.k1 = ksteps;
            s.whole = true;
            return true;
        }
        if (u0 >= u) return false;
        const long long tl = u0 / ksteps, ts = tl * ksteps;
        place(whole_tiles + static_cast<int>(tl), s);
        s.k0 = static_cast<int>(u0 - ts);
        s.k1 = static_cast<int>((u < ts + ksteps ? u : ts + ksteps) - ts);
        s.whole = s.k0 == 0 && s.k1 == ksteps;
        if (!s.whole) {
            s.first = owner(ts);
            s.last = owner(ts + ksteps - 1);
        }
        u0 = ts + s.k1;
        return true;
    }
};

__device__ __forceinline__ bool f8_wait(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *status) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > kF8WaitLimit) {
            *abort = 1;
            atomicOr(status, kStatusF8Timeout);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ uint32_t in_even_cta(uint32_t addr) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(addr));
    return remote;
}

__device__ __forceinline__ void arrive_cluster(uint32_t remote) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// K-major operand of 128-byte rows in the 128-byte swizzle: groups of eight rows
// 1024 bytes apart; 32 values on along K are 32 bytes on.
__device__ __forceinline__ uint64_t f8_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// sixteen lanes' 32 columns: for each eight of them the fragment of a 16 x 8 tile
// (lane t: rows t / 4 and t / 4 + 8, columns 2 (t % 4) and the next)
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ uint64_t pair64(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t pair64(float lo, float hi) {
    return pair64(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float2 floats(uint64_t v) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void fma2(uint64_t &c, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

template <class P>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P::THREADS, 1)
k_linear_f8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const F8Params p) {
    constexpr int NT = P::NT, DRAIN = P::DRAIN, STAGES = P::STAGES, ACCS = P::ACCS, SCALES = P::SCALES;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + P::OFF_BARS);
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_sh;
    __shared__ int total_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
    const uint32_t acc_full0 = empty0 + 8 * STAGES, acc_empty0 = acc_full0 + 8 * ACCS;
    const uint32_t sc_full0 = acc_empty0 + 8 * ACCS, sc_empty0 = sc_full0 + 8 * SCALES;
    const uint32_t done = sc_empty0 + 8 * SCALES;

    if (threadIdx.x == 0) {
        auto init = [](uint32_t bar, uint32_t n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n));
        };
        for (int s = 0; s < STAGES; ++s) {
            init(full0 + 8 * s, 1);                 // used in the even CTA: its expected bytes cover both
            init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < ACCS; ++a) {
            init(acc_full0 + 8 * a, 1);
            init(acc_empty0 + 8 * a, 2 * DRAIN);    // used in the even CTA: both CTAs' drain warps
        }
        for (int s = 0; s < SCALES; ++s) {
            init(sc_full0 + 8 * s, 32);
            init(sc_empty0 + 8 * s, DRAIN);
        }
        init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_sh = 0;
    }
    // the list of experts: a range that is out of order is empty
    int *row0 = reinterpret_cast<int *>(smem + P::OFF_LIST), *rows = row0 + p.experts + 1, *tiles = rows + p.experts + 1;
    if (warp == 0) {
        if (p.offsets == nullptr) {
            if (lane == 0) {
                row0[0] = 0;
                rows[0] = static_cast<int>(p.M);
                tiles[0] = 0;
                tiles[1] = total_sh = static_cast<int>((p.M + NT - 1) / NT);
            }
        } else {
            int sum = 0, most = INT32_MIN;
            bool bad = false;
            for (int e0 = 0; e0 < p.experts; e0 += 32) {
                const int e = e0 + lane;
                const bool in = e < p.experts;
                const int a = in ? p.offsets[e] : INT32_MIN, b = in ? p.offsets[e + 1] : INT32_MIN;
                int top = a, t = 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, top, o);
                    if (lane >= o) top = max(top, v);
                }
                top = max(top, most);               // the largest offset so far
                const bool ok = a >= 0 && b >= a && b <= p.M && a >= top;
                const int n = in && ok ? b - a : 0;
                bad |= in && !ok;
                t = (n + NT - 1) / NT;
                int s = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, s, o);
                    if (lane >= o) s += v;
                }
                if (in) {
                    row0[e] = a;
                    rows[e] = n;
                    tiles[e] = sum + s - t;
                }
                sum += __shfl_sync(0xffffffffu, s, 31);
                most = __shfl_sync(0xffffffffu, top, 31);
            }
            if (bad) atomicOr(p.status, kStatusIndex);
            if (lane == 0) tiles[p.experts] = total_sh = sum;
        }
    }
    if (warp == DRAIN) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_base_sh)), "r"(static_cast<uint32_t>(P::TMEM)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync_all();   // barriers of both CTAs initialised, TMEM allocated
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_base_sh;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const F8List list{row0, rows, tiles, p.experts, total_sh};

    if (warp >= DRAIN) {
        if constexpr (P::WIDE) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == DRAIN) {
            // -------------------------------------------- MMA issue (even CTA, one thread)
            if (rank == 0 && lane == 0) {
                uint32_t it = 0;
                F8Iter<NT> iter(list, p, pair, pairs);
                F8Seg sg;
                while (!abort_sh && iter.next(sg)) {
                    // D fp32, A and B e4m3, K-major, M = 256
                    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(sg.mma_n >> 3) << 17) | (16u << 24);
                    for (int ks = sg.k0; ks < sg.k1; ++ks, ++it) {
                        const int s = it % STAGES, a = it % ACCS;
                        if (!f8_wait(acc_empty0 + 8 * a, ((it / ACCS) & 1) ^ 1, &abort_sh, p.status)) break;
                        if (!f8_wait(full0 + 8 * s, (it / STAGES) & 1, &abort_sh, p.status)) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t w = smem_u32(smem + s * P::STAGE);
                        const uint64_t wd = f8_desc(w), xd = f8_desc(w + kWBytes);
#pragma unroll
                        for (int kk = 0; kk < kStepK / 32; ++kk)
                            asm volatile(
                                "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                                "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                                ::"r"(tmem + static_cast<uint32_t>(NT * a)), "l"(wd + 2 * kk), "l"(xd + 2 * kk),
                                  "r"(idesc), "r"(kk > 0 ? 1u : 0u));
                        auto commit = [](uint32_t bar) {
                            asm volatile(
                                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
                                ".b64 [%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
                        };
                        commit(empty0 + 8 * s);
                        commit(acc_full0 + 8 * a);
                    }
                }
                // let every issued MMA finish before the pair's TMEM is released
                if (it > 0) {
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                                 ::"r"(done) : "memory");
                    const long long t0 = clock64();
                    while (!mbar_try(done, 0) && clock64() - t0 < kF8WaitLimit) {
                    }
                }
            }
        } else if (warp == DRAIN + 1) {
            // -------------------------------------------- tensor copies
            if (lane == 0) {
                uint32_t it = 0;
                F8Iter<NT> iter(list, p, pair, pairs);
                F8Seg sg;
                while (!abort_sh && iter.next(sg)) {
                    const int n0 = sg.ntile * 2 * kRowsW;
                    const int boxes = (sg.mma_n / 2 + kBoxRows - 1) / kBoxRows;
                    // weight rows past N are not loaded (what they multiply is not stored)
                    const bool mine = n0 + static_cast<int>(rank) * kRowsW < p.N;
                    const uint32_t bytes =
                        2 * boxes * kBoxRows * kStepK + (n0 + kRowsW < p.N ? 2 * kWBytes : kWBytes);
                    const int wrow = sg.e * p.N + n0 + static_cast<int>(rank) * kRowsW;
                    const int xrow = sg.m0 + static_cast<int>(rank) * (sg.mma_n / 2);
                    for (int ks = sg.k0; ks < sg.k1; ++ks, ++it) {
                        const int s = it % STAGES;
                        if (!f8_wait(empty0 + 8 * s, ((it / STAGES) & 1) ^ 1, &abort_sh, p.status)) break;
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                                         ::"r"(full0 + 8 * s), "r"(bytes) : "memory");
                        const uint32_t bar = in_even_cta(full0 + 8 * s);
                        const uint32_t w = smem_u32(smem + s * P::STAGE);
                        auto copy = [&](uint32_t dst, const CUtensorMap *map, int row) {
                            asm volatile(
                                "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx"
                                "::bytes [%0], [%1, {%2, %3}], [%4];"
                                ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(ks * kStepK), "r"(row), "r"(bar)
                                : "memory");
                        };
                        if (mine) copy(w, &tmW, wrow);
                        for (int b = 0; b < boxes; ++b)
                            copy(w + kWBytes + b * kBoxRows * kStepK, &tmX, xrow + b * kBoxRows);
                    }
                }
                // after a wait ran out: the copies in flight land before the pair leaves
                if (abort_sh && rank == 0)
                    for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j) {
                        const long long t0 = clock64();
                        while (!mbar_try(full0 + 8 * (j % STAGES), (j / STAGES) & 1) &&
                               clock64() - t0 < kF8WaitLimit / 16) {
                        }
                    }
            }
        } else if (warp == DRAIN + 2) {
            // -------------------------------------------- the tokens' scales
            // column c of a tile at ((c / 16) * 4 + (c % 8) / 2) * 4 + (c / 8 % 2) * 2 + c % 2: the four
            // that a lane of a fragment needs of sixteen columns lie together
            uint32_t it = 0;
            F8Iter<NT> iter(list, p, pair, pairs);
            F8Seg sg;
            while (!abort_sh && iter.next(sg)) {
                for (int ks = sg.k0; ks < sg.k1; ++ks, ++it) {
                    const int s = it % SCALES;
                    if (!f8_wait(sc_empty0 + 8 * s, ((it / SCALES) & 1) ^ 1, &abort_sh, p.status)) break;
                    const uint32_t to = smem_u32(smem + P::OFF_SCALES) + s * NT * 4;
                    const float *from = p.sx + static_cast<int64_t>(ks) * p.M + sg.m0;
#pragma unroll
                    for (int i = 0; i < NT / 32; ++i) {
                        const int c = lane + 32 * i;
                        const int at = ((c >> 4) * 4 + ((c & 7) >> 1)) * 4 + ((c >> 3) & 1) * 2 + (c & 1);
                        if (c < sg.cols)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + at * 4), "l"(from + c)
                                         : "memory");
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sc_full0 + 8 * s)
                                 : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        __syncwarp();
    } else {
        if constexpr (P::WIDE) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ------------------------------------------------ drain
        constexpr int GROUPS = P::COLS / 32;             // 32 tokens at a time
        const int q = warp & 3, c0 = (warp >> 2) * P::COLS;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t acc_empty_even = in_even_cta(acc_empty0);
        const float *ring = reinterpret_cast<const float *>(smem + P::OFF_SCALES);
        uint32_t it = 0;
        F8Iter<NT> iter(list, p, pair, pairs);
        F8Seg sg;
        // the warp acts as one: a lane that saw an abort takes the others along
        while (__all_sync(0xffffffffu, !abort_sh) && iter.next(sg)) {
            const int n0 = sg.ntile * 2 * kRowsW + static_cast<int>(rank) * kRowsW;
            const float *sw = p.sw + (static_cast<int64_t>(sg.e) * p.nblocks + n0 / kRowsW) * p.ksteps;
            const bool some = n0 < p.N;                  // this CTA has columns of the tile
            const int groups = min(GROUPS, (sg.cols - c0 + 31) / 32);     // those with tokens (none: <= 0)
            uint64_t acc[GROUPS][16];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[g][i] = 0ull;
            float next = some ? __ldg(sw + sg.k0) : 0.0f;
            int ks = sg.k0;
            for (; ks < sg.k1; ++ks, ++it) {
                const int s = it % SCALES, a = it % ACCS;
                const uint64_t w2 = pair64(next, next);
                if (some && ks + 1 < sg.k1) next = __ldg(sw + ks + 1);
                if (!__all_sync(0xffffffffu, f8_wait(sc_full0 + 8 * s, (it / SCALES) & 1, &abort_sh, p.status) &&
                                                 f8_wait(acc_full0 + 8 * a, (it / ACCS) & 1, &abort_sh, p.status)))
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    if (g >= groups) break;
                    uint32_t v[2][16];
                    const uint32_t at = tmem + lanes + static_cast<uint32_t>(NT * a + c0 + 32 * g);
                    tmem_ld_16x32(at, v[0]);
                    tmem_ld_16x32(at + (16u << 16), v[1]);
                    uint64_t f[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 x = *reinterpret_cast<const float4 *>(
                            ring + s * NT + (((c0 + 32 * g) >> 4) + j) * 16 + (lane & 3) * 4);
                        f[2 * j] = mul2(pair64(x.x, x.y), w2);
                        f[2 * j + 1] = mul2(pair64(x.z, x.w), w2);
                    }
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            fma2(acc[g][h * 8 + i * 2], pair64(v[h][4 * i], v[h][4 * i + 1]), f[i]);
                            fma2(acc[g][h * 8 + i * 2 + 1], pair64(v[h][4 * i + 2], v[h][4 * i + 3]), f[i]);
                        }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    arrive_cluster(acc_empty_even + 8 * a);
                    mbar_arrive_local(sc_empty0 + 8 * s);
                }
            }
            if (ks < sg.k1) break;                       // a wait ran out
            if (!some || groups <= 0) continue;          // nothing of the tile is this warp's
            if (!sg.whole) {
                // store the part; the warp that comes last adds all parts in order
                auto slot = [&](int w) {
                    return reinterpret_cast<uint64_t *>(
                               p.slots + (static_cast<int64_t>(w) * 4 + (w == sg.first ? 2 : 0) + rank) * P::SLOT) +
                           static_cast<int64_t>(warp) * GROUPS * 16 * 32 + lane;
                };
                uint64_t *to = slot(pair);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    if (g < groups)
#pragma unroll
                        for (int i = 0; i < 16; ++i) __stcg(reinterpret_cast<unsigned long long *>(to + (g * 16 + i) * 32), acc[g][i]);
                __threadfence();
                __syncwarp();
                unsigned int *counter = p.counters + (sg.first * 2 + static_cast<int>(rank)) * kF8MaxDrain + warp;
                unsigned int before = 0;
                if (lane == 0) before = atomicAdd(counter, 1u);
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before != static_cast<unsigned int>(sg.last - sg.first)) continue;
                __threadfence();
                if (lane == 0) *counter = 0u;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    if (g < groups) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[g][i] = 0ull;
                        for (int w = sg.first; w <= sg.last; ++w) {
                            const uint64_t *from = slot(w) + g * 16 * 32;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                acc[g][i] = add2(acc[g][i], __ldcg(reinterpret_cast<const unsigned long long *>(from + i * 32)));
                        }
                    }
            }
            // ---- Y: a lane's fragments are two tokens (columns of the tile) by one weight row
            const int nb = n0 + q * 32;                  // this warp's 32 columns of Y
            if (p.ytype == 0) {
                float *Y = static_cast<float *>(p.Y);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    if (g < groups)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int c = c0 + 32 * g + ((i >> 1) & 3) * 8 + (lane & 3) * 2;
                            const int n = nb + (i >> 3) * 16 + (i & 1) * 8 + (lane >> 2);
                            const float2 v = floats(acc[g][i]);
                            if (n < p.N) {
                                float *y = Y + (static_cast<int64_t>(sg.m0) + c) * p.ldy + n;
                                if (c < sg.cols) *y = v.x;
                                if (c + 1 < sg.cols) y[p.ldy] = v.y;
                            }
                        }
            } else {
                // sixteen tokens at a time through shared memory, turned on the way in
                uint16_t *Y = static_cast<uint16_t *>(p.Y);
                unsigned char *turn = smem + P::OFF_OUT + warp * P::OUT_ROWS * P::OUT_PITCH;
                const uint32_t put = smem_u32(turn) + (lane & 7) * P::OUT_PITCH + (lane >> 3) * 16;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    if (g < groups)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            __syncwarp();
#pragma unroll
                            for (int ii = 0; ii < 2; ++ii) {
                                uint32_t b[4];           // weight rows 0-7, 8-15, 16-23, 24-31
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float2 v = floats(acc[g][(j >> 1) * 8 + (hh * 2 + ii) * 2 + (j & 1)]);
                                    b[j] = f32_to_bf16_bits(v.x) | (static_cast<uint32_t>(f32_to_bf16_bits(v.y)) << 16);
                                }
                                asm volatile(
                                    "stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                                    ::"r"(put + ii * 8 * P::OUT_PITCH), "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
                                    : "memory");
                            }
                            __syncwarp();
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const int row = r * 8 + (lane >> 2), c = c0 + 32 * g + hh * 16 + row;
                                const int n = nb + (lane & 3) * 8;
                                if (c >= sg.cols || n >= p.N) continue;
                                const uint4 v = *reinterpret_cast<const uint4 *>(turn + row * P::OUT_PITCH + (lane & 3) * 16);
                                uint16_t *y = Y + (static_cast<int64_t>(sg.m0) + c) * p.ldy + n;
                                if (p.vec && n + 8 <= p.N) {
                                    *reinterpret_cast<uint4 *>(y) = v;
                                } else {
                                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                                    for (int j = 0; j < 8 && n + j < p.N; ++j)
                                        y[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
                                }
                            }
                        }
            }
        }
    }
    // nobody leaves while the peer may still arrive on this CTA's barriers or while
    // MMAs of the pair are in flight (the even CTA waited for them above)
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync_all();
    if (warp == DRAIN) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(static_cast<uint32_t>(P::TMEM)));
    }
}

constexpr size_t kF8CounterBytes(int pairs) {
    return (static_cast<size_t>(pairs) * 2 * kF8MaxDrain * 4 + 255) / 256 * 256;
}

template <int NT>
tq_status launch_f8(const F8Product &f, const DeviceInfo &dev, cudaStream_t s) {
    using P = F8Plan<NT>;
    auto kern = k_linear_f8<P>;
    if (dev.id < 0 || dev.id >= 64 || dev.sms < 2) return TQ_ERR_DEVICE;
    static bool configured[64] = {false};
    if (!configured[dev.id]) {
        cudaFuncAttributes at;
        cudaError_t e = cudaFuncGetAttributes(&at, kern);
        if (e != cudaSuccess) return cuda_fail(e);
        // the warps' own register counts have to be covered by the launch's
        if (P::WIDE && at.numRegs * P::THREADS < 216 * 256 + 72 * 128) return TQ_ERR_DEVICE;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P::smem(TQ_MAX_EXPERTS));
        if (e != cudaSuccess) return cuda_fail(e);
        configured[dev.id] = true;
    }
    F8Params p{};
    p.sx = f.sx;
    p.M = f.M;
    p.offsets = f.offsets;
    p.experts = static_cast<int>(f.offsets ? f.experts : 1);
    p.sw = f.sw;
    p.N = static_cast<int>(f.N);
    p.ksteps = static_cast<int>((f.K + kStepK - 1) / kStepK);
    p.nblocks = static_cast<int>((f.N + kRowsW - 1) / kRowsW);
    p.ntiles = static_cast<int>((f.N + 2 * kRowsW - 1) / (2 * kRowsW));
    p.Y = f.Y;
    p.ldy = f.ldy;
    p.ytype = f.ytype;
    p.vec = (reinterpret_cast<uintptr_t>(f.Y) & 15) == 0 && f.ldy % 8 == 0 ? 1 : 0;
    p.status = status_word();
    if (!p.status) return TQ_ERR_DEVICE;
    const int most = dev.sms / 2;
    p.counters = static_cast<unsigned int *>(f.ws);
    p.slots = static_cast<unsigned char *>(f.ws) + kF8CounterBytes(most);
    p.min_steps = 2;
    CUtensorMap tmW, tmX;
    if (!make_map_u8(&tmW, f.Wq, p.experts * f.N, f.K, kStepK, kRowsW, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_u8(&tmX, f.Xq, f.M, f.K, kStepK, kBoxRows, CU_TENSOR_MAP_SWIZZLE_128B))
        return TQ_ERR_DEVICE;
    // token tiles there may be: one more an expert than whole ones
    const int64_t token_tiles = f.M / NT + (f.M < p.experts ? f.M : p.experts);
    if (token_tiles * p.ntiles > (1ll << 30)) return TQ_ERR_OVERFLOW;
    const int64_t steps = token_tiles * p.ntiles * p.ksteps;
    const int64_t pairs = steps / p.min_steps < 1 ? 1 : (steps / p.min_steps < most ? steps / p.min_steps : most);
    kern<<<static_cast<unsigned>(2 * pairs), P::THREADS, P::smem(p.experts), s>>>(tmW, tmX, p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace

// counters, then two parts of a tile a CTA
size_t f8_workspace_bytes(const DeviceInfo &dev) {
    const int pairs = dev.sms / 2;
    return kF8CounterBytes(pairs) + static_cast<size_t>(pairs) * 4 * F8Plan<256>::SLOT;
}

// Few tokens an expert: tiles of 64, more of the weights in flight.
tq_status launch_linear_f8(const F8Product &p, const DeviceInfo &dev, cudaStream_t s) {
    const int64_t experts = p.offsets ? p.experts : 1;
    return p.M <= 64 * experts ? launch_f8<64>(p, dev, s) : launch_f8<256>(p, dev, s);
}

}  // namespace tq
