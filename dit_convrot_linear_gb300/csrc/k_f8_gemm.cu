// The product of 8-bit floating-point operands with a scale for each block of 128,
//   Y[m][n] = sum_b sx[b][m] * sw[n / 128][b] * sum_{k in block b} xq[m][k] * wq[n][k],
// of one matrix, or of one matrix an expert over rows sorted by expert, on tcgen05
// (kind::f8f6f4: e4m3 operands as they are, at twice the rate of fp16).
//
// A pair of CTAs (tcgen05 cta_group::2) computes 256 output columns (weight rows) of
// up to NT tokens.  A step of K is one scale block, four MMAs of 32; the accumulator
// of each step lies in TMEM of its own, and the drain warps add it, times its scales,
// to the sums in their registers.  Two forms:
//   many tokens  (NT = 256) the tokens are the MMA's M side, so that a TMEM lane is
//                a token and a step's scales are one number a thread,
//                acc += (sx[b][token] * sw[block][b]) * part;
//   few tokens   (NT = 64) the weights are the M side and the tokens the N side, in
//                steps of 16: an expert's few rows cost no empty rows of a 128-row
//                tile.  The scales differ from column to column and come from shared
//                memory; that takes 4 bytes a lane and value, 1024 cycles a step at 256
//                tokens, and is hidden behind the weights' stream at 64.
// Per CTA:
//   drain warps  (a TMEM lane quarter each; with eight of them two a quarter, half
//                the columns each) multiply and add, and write Y;
//   MMA warp     allocates TMEM for the pair; in the even CTA one thread issues;
//   copy warp    tensor copies of both operands into the ring (128-byte swizzle);
//   scale warp   each step's scales, sx * sw, into shared memory.
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

constexpr int kHalf = 128;                // rows a CTA brings to the M side: half a pair's
constexpr int kTileN = 256;               // weight rows (columns of Y) of a tile
constexpr int kStepK = 128;               // K of a step: one scale block
constexpr int kABytes = kHalf * kStepK;   // a stage's M side
constexpr long long kF8WaitLimit = 4000000000ll;   // clock cycles, about 2 s
constexpr unsigned int kStatusF8Timeout = 64u;

template <int NT_>
struct F8Plan {
    static constexpr int NT = NT_;
    static constexpr bool WIDE = NT == 256;                    // tokens on the M side
    static constexpr int NCOLS = WIDE ? kTileN : NT;           // columns of an accumulator: the N side
    static constexpr int COLS = WIDE ? 128 : 64;               // columns a drain warp
    static constexpr int DRAIN = 4 * NCOLS / COLS;             // drain warps
    // many tokens: a step's columns are two accumulators of 128, each with its own MMAs, so
    // that one is filled while the other is drained
    static constexpr int HALVES = WIDE ? 2 : 1;
    static constexpr int ISSUERS = 2 * HALVES;                 // MMA warps: the steps in turn, a half each
    static constexpr int OTHERS = WIDE ? 8 : 4;                // warps that do not drain
    static constexpr int THREADS = (DRAIN + OTHERS) * 32;
    static constexpr int B_BOX = WIDE ? 64 : 32;               // rows of one tensor copy of the N side
    static constexpr int B_BYTES = NCOLS / 2 * kStepK;
    static constexpr int STAGE = kABytes + B_BYTES;
    static constexpr int STAGES = WIDE ? 6 : 10;
    static constexpr int TURNS = WIDE ? 2 : 4;                 // steps with accumulators in TMEM
    static constexpr int ACCS = TURNS * HALVES, ACC_COLS = NCOLS / HALVES;
    static constexpr int TMEM = ACC_COLS * ACCS;
    static constexpr int SCALES = WIDE ? 256 : NT;             // scales of a step: a slot for each turn
    static constexpr int OFF_SCALES = STAGES * STAGE;
    static constexpr int OUT_BYTES = WIDE ? DRAIN * 32 * 64 : 0;   // 64 bytes of 32 rows a warp
    static constexpr int OFF_OUT = OFF_SCALES + TURNS * SCALES * 4;
    static constexpr int OFF_BARS = OFF_OUT + OUT_BYTES;
    static constexpr int NBARS = 2 * STAGES + 2 * ACCS + TURNS + 1;
    static constexpr int OFF_LIST = OFF_BARS + (NBARS * 8 + 15) / 16 * 16;
    // the list of experts: first row, rows, tiles before
    static constexpr int smem(int64_t experts) { return OFF_LIST + static_cast<int>(experts + 1) * 12 + 16; }
    static constexpr int SLOT = DRAIN * 32 * (COLS / 2) * 8;   // bytes of a CTA's partial tile
};
static_assert(F8Plan<256>::smem(TQ_MAX_EXPERTS) <= 226 * 1024 && F8Plan<64>::smem(TQ_MAX_EXPERTS) <= 226 * 1024,
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
    int ytype, vec;                      // vec: rows of Y allow 16-byte stores (few tokens: 4-byte ones)
    unsigned int *status;
    unsigned int *counters;              // [pairs][2 CTAs][kF8MaxDrain]
    unsigned char *slots;                // [pairs][2][2 CTAs][SLOT]
    int min_steps;                       // K steps a pair takes of split tiles, at least
};

// A piece of work: the tile's place, K steps k0 .. k1 - 1, and for a piece of a
// split tile the pairs that have its first and last step.
struct F8Seg {
    int e, ntile, m0, cols, k0, k1;      // cols: tokens of the tile (at most NT)
    bool whole;
    int first, last;
};

// The list of work, in shared memory: of each expert its first row, its rows and the
// token tiles before it (one more entry), and how the tiles are cut.
struct F8Cut {
    int tiles;       // tiles in all
    int whole;       // of them computed whole
    int units;       // K steps of the others,
    int use;         // shared by this many pairs
};

// The pieces of work of a pair, in order.  (What does not change lies in shared
// memory: the drain warps have few registers to spare.)
struct F8Iter {
    int i, u0;
    __device__ F8Iter(const F8Cut &c, int pair) : i(0), u0(pair < c.use ? c.units * pair / c.use : 0) {}
    // the pair whose steps include x
    static __device__ int owner(const F8Cut &c, int x) {
        int q = x * c.use / c.units;
        while (q + 1 < c.use && c.units * (q + 1) / c.use <= x) ++q;
        while (q > 0 && c.units * q / c.use > x) --q;
        return q;
    }
    static __device__ void place(const int *list, const F8Params &p, int tile, F8Seg &s) {
        const int *row0 = list, *rows = list + p.experts + 1, *tiles = rows + p.experts + 1;
        int lo = 0, hi = p.experts;      // tiles[lo] * ntiles <= tile < tiles[hi] * ntiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tiles[mid] * p.ntiles <= tile) lo = mid; else hi = mid;
        }
        const int at = tile - tiles[lo] * p.ntiles, parts = tiles[lo + 1] - tiles[lo];
        const int n = rows[lo], each = ((n + parts - 1) / parts + 15) / 16 * 16;
        const int part = at % parts;
        s.e = lo;
        s.ntile = at / parts;
        s.m0 = row0[lo] + part * each;
        s.cols = min(each, n - part * each);
    }
    __device__ bool next(const F8Cut &c, const int *list, const F8Params &p, F8Seg &s) {
        const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, ksteps = p.ksteps;
        const int t = pair + i * pairs;
        if (t < c.whole) {
            ++i;
            place(list, p, t, s);
            s.k0 = 0;
            s.k1 = ksteps;
            s.whole = true;
            return true;
        }
        const int u1 = pair < c.use ? c.units * (pair + 1) / c.use : 0;
        if (u0 >= u1) return false;
        const int tl = u0 / ksteps, ts = tl * ksteps;
        place(list, p, c.whole + tl, s);
        s.k0 = u0 - ts;
        s.k1 = min(u1, ts + ksteps) - ts;
        s.whole = s.k0 == 0 && s.k1 == ksteps;
        s.first = s.last = pair;
        if (!s.whole) {
            s.first = owner(c, ts);
            s.last = owner(c, ts + ksteps - 1);
        }
        u0 = ts + s.k1;
        return true;
    }
};

// What these barriers hand over is shared memory filled by tensor copies, this CTA's
// own stores and TMEM: an acquire at CTA scope is enough.
__device__ __forceinline__ bool f8_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool f8_wait(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *status) {
    if (f8_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!f8_try(bar, parity)) {
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

// What it hands over is TMEM that has been read (tcgen05.wait::ld came before), no
// memory: a release at cluster scope would wait for everything this thread has in
// flight (2000 cycles a step).
__device__ __forceinline__ void arrive_cluster(uint32_t remote) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// K-major operand of 128-byte rows in the 128-byte swizzle: groups of eight rows
// 1024 bytes apart; 32 values on along K are 32 bytes on.
__device__ __forceinline__ uint64_t f8_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Waits for what tmem_ld32 has asked for; the operands tie the values' uses to the
// wait without holding back other loads.
__device__ __forceinline__ void tmem_wait32(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]));
    asm volatile("" : "+r"(v[30]), "+r"(v[31]));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <class P>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P::THREADS, 1)
k_linear_f8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const F8Params p) {
    constexpr int NT = P::NT, DRAIN = P::DRAIN, STAGES = P::STAGES, ACCS = P::ACCS, TURNS = P::TURNS, HALVES = P::HALVES;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + P::OFF_BARS);
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_sh;
    __shared__ F8Cut cut;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
    const uint32_t acc_full0 = empty0 + 8 * STAGES, acc_empty0 = acc_full0 + 8 * ACCS;
    const uint32_t sc_empty0 = acc_empty0 + 8 * ACCS, done = sc_empty0 + 8 * TURNS;

    if (threadIdx.x == 0) {
        auto init = [](uint32_t bar, uint32_t n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n));
        };
        for (int s = 0; s < STAGES; ++s) {
            init(full0 + 8 * s, 1);                 // used in the even CTA: its expected bytes cover both
            init(empty0 + 8 * s, HALVES);
        }
        for (int a = 0; a < ACCS; ++a) {
            init(acc_full0 + 8 * a, 2);             // the step's MMAs, and its scales
            init(acc_empty0 + 8 * a, 2 * DRAIN / HALVES);   // used in the even CTA: both CTAs' drain warps
        }
        for (int s = 0; s < TURNS; ++s) init(sc_empty0 + 8 * s, DRAIN);   // a step's scales have been read
        init(done, P::ISSUERS);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_sh = 0;
    }
    // the list of experts: a range that is out of order is empty
    const int *list = reinterpret_cast<const int *>(smem + P::OFF_LIST);
    if (warp == 0) {
        int *row0 = reinterpret_cast<int *>(smem + P::OFF_LIST), *rows = row0 + p.experts + 1, *tiles = rows + p.experts + 1;
        int total = static_cast<int>((p.M + NT - 1) / NT);       // token tiles
        if (p.offsets == nullptr) {
            if (lane == 0) {
                row0[0] = 0;
                rows[0] = static_cast<int>(p.M);
                tiles[0] = 0;
                tiles[1] = total;
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
            if (lane == 0) tiles[p.experts] = sum;
            total = sum;
        }
        if (lane == 0) {
            // the last round of tiles is split where it would leave a good part of the pairs idle
            const int n = total * p.ntiles, pairs = gridDim.x >> 1, rest = n % pairs;
            const bool split = rest > 0 && rest * 100 < pairs * 85;
            cut.tiles = n;
            cut.whole = split ? n - rest : n;
            cut.units = split ? rest * p.ksteps : 0;
            cut.use = max(1, min(pairs, cut.units / p.min_steps));
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
    const int pair = blockIdx.x >> 1;

    if (warp >= DRAIN) {
        if constexpr (P::WIDE) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // columns of accumulator h of a tile: tokens, or weight rows, rounded up to 16 (one
        // without any still takes part, and nothing of it is stored)
        auto mma_n = [&](const F8Seg &sg, int h) {
            const int n = P::WIDE ? min(P::ACC_COLS, p.N - sg.ntile * kTileN - h * P::ACC_COLS) : sg.cols;
            return (max(n, 1) + 15) / 16 * 16;
        };
        if (warp < DRAIN + P::ISSUERS) {
            // -------------------------------------------- MMA issue (even CTA, one thread a warp)
            // A step's waits, commits and issues take one thread 800 cycles, its MMAs 512.
            if (rank == 0 && lane == 0) {
                const int h = (warp - DRAIN) % HALVES;
                const uint32_t turn = (warp - DRAIN) / HALVES;
                uint32_t it = 0;
                F8Iter iter(cut, pair);
                F8Seg sg;
                while (!abort_sh && iter.next(cut, list, p, sg)) {
                    // D fp32, A and B e4m3, K-major, M = 256
                    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(mma_n(sg, h) >> 3) << 17) | (16u << 24);
                    for (int ks = sg.k0; ks < sg.k1; ++ks, ++it) {
                        if ((it & 1) != turn) continue;
                        const int s = it % STAGES, a = (it % TURNS) * HALVES + h;
                        if (!f8_wait(full0 + 8 * s, (it / STAGES) & 1, &abort_sh, p.status)) break;
                        if (!f8_wait(acc_empty0 + 8 * a, ((it / TURNS) & 1) ^ 1, &abort_sh, p.status)) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t at = smem_u32(smem + s * P::STAGE);
                        const uint64_t ad = f8_desc(at), bd = f8_desc(at + kABytes + h * P::B_BOX * kStepK);
#pragma unroll
                        for (int kk = 0; kk < kStepK / 32; ++kk)
                            asm volatile(
                                "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                                "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                                ::"r"(tmem + static_cast<uint32_t>(P::ACC_COLS * a)), "l"(ad + 2 * kk), "l"(bd + 2 * kk),
                                  "r"(idesc), "r"(kk > 0 ? 1u : 0u));
                        auto commit = [](uint32_t bar) {
                            asm volatile(
                                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
                                ".b64 [%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
                        };
                        commit(acc_full0 + 8 * a);
                        commit(empty0 + 8 * s);
                    }
                }
                // let every issued MMA finish before the pair's TMEM is released
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                             ::"r"(done) : "memory");
                const long long t0 = clock64();
                while (!f8_try(done, 0) && clock64() - t0 < kF8WaitLimit) {
                }
            }
        } else if (warp == DRAIN + P::ISSUERS) {
            // -------------------------------------------- tensor copies
            if (lane == 0) {
                uint32_t it = 0;
                F8Iter iter(cut, pair);
                F8Seg sg;
                while (!abort_sh && iter.next(cut, list, p, sg)) {
                    // rows of the M side that are past the tile's are not loaded (what comes of
                    // them is not stored); the N side is copied in whole boxes, which hold half
                    // of an accumulator's columns in each CTA
                    const int n0 = sg.ntile * kTileN;
                    const int wrow = sg.e * p.N + n0;
                    const int rows_a = P::WIDE ? sg.cols : p.N - n0;
                    const int halves = HALVES == 2 && p.N - n0 > P::ACC_COLS ? 2 : 1;
                    const bool mine = static_cast<int>(rank) * kHalf < rows_a;
                    const uint32_t bytes =
                        2 * halves * P::B_BOX * kStepK + (kHalf < rows_a ? 2 * kABytes : kABytes);
                    const int arow = (P::WIDE ? sg.m0 : wrow) + static_cast<int>(rank) * kHalf;
                    for (int ks = sg.k0; ks < sg.k1; ++ks, ++it) {
                        const int s = it % STAGES;
                        if (!f8_wait(empty0 + 8 * s, ((it / STAGES) & 1) ^ 1, &abort_sh, p.status)) break;
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                                         ::"r"(full0 + 8 * s), "r"(bytes) : "memory");
                        const uint32_t bar = in_even_cta(full0 + 8 * s);
                        const uint32_t at = smem_u32(smem + s * P::STAGE);
                        auto copy = [&](uint32_t dst, const CUtensorMap *map, int row) {
                            asm volatile(
                                "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx"
                                "::bytes [%0], [%1, {%2, %3}], [%4];"
                                ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(ks * kStepK), "r"(row), "r"(bar)
                                : "memory");
                        };
                        if (mine) copy(at, &tmA, arow);
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            if (h < halves)
                                copy(at + kABytes + h * P::B_BOX * kStepK, &tmB,
                                     (P::WIDE ? wrow + h * P::ACC_COLS : sg.m0) + static_cast<int>(rank) * (mma_n(sg, h) / 2));
                    }
                }
                // after a wait ran out: the copies in flight land before the pair leaves
                if (abort_sh && rank == 0)
                    for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j) {
                        const long long t0 = clock64();
                        while (!f8_try(full0 + 8 * (j % STAGES), (j / STAGES) & 1) &&
                               clock64() - t0 < kF8WaitLimit / 16) {
                        }
                    }
            }
        } else if (warp == DRAIN + P::ISSUERS + 1) {
            // -------------------------------------------- scales
            // Each step's sx * sw into its turn's slot, loaded AHEAD steps before.  Many
            // tokens: 128 of this CTA's tokens with the first scale block of columns, then with
            // the second.  Few: each token with this CTA's block.  (Places past the tile's rows or
            // N take their last one's; what comes of them is not stored.)
            constexpr int AHEAD = 4, EACH = P::WIDE ? 4 : NT / 32, BLOCKS = P::WIDE ? 2 : 1;
            uint32_t it = 0;
            F8Iter iter(cut, pair);
            F8Seg sg;
            while (__all_sync(0xffffffffu, !abort_sh) && iter.next(cut, list, p, sg)) {
                const int n0 = sg.ntile * kTileN + (P::WIDE ? 0 : static_cast<int>(rank) * kHalf);
                const int t0 = P::WIDE ? static_cast<int>(rank) * kHalf : 0;
                const float *sx[EACH], *sw[BLOCKS];
#pragma unroll
                for (int i = 0; i < EACH; ++i)
                    sx[i] = p.sx + sg.k0 * p.M + sg.m0 + min(t0 + lane + 32 * i, sg.cols - 1);
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j)
                    sw[j] = p.sw + (static_cast<int64_t>(sg.e) * p.nblocks + min(n0 / 128 + j, p.nblocks - 1)) * p.ksteps;
                float x[AHEAD][EACH], w[AHEAD][BLOCKS];
                auto load = [&](int ks, float (&xs)[EACH], float (&ws)[BLOCKS]) {
                    if (ks >= sg.k1) return;
#pragma unroll
                    for (int i = 0; i < EACH; ++i) {
                        xs[i] = __ldg(sx[i]);
                        sx[i] += p.M;
                    }
#pragma unroll
                    for (int j = 0; j < BLOCKS; ++j) ws[j] = __ldg(sw[j] + ks);
                };
#pragma unroll
                for (int d = 0; d < AHEAD; ++d) load(sg.k0 + d, x[d], w[d]);
                bool ok = true;
                for (int ks = sg.k0; ok && ks < sg.k1; ks += AHEAD)
#pragma unroll
                    for (int d = 0; d < AHEAD; ++d) {
                        if (!ok || ks + d >= sg.k1) break;
                        const int s = it % TURNS;
                        ok = __all_sync(0xffffffffu, f8_wait(sc_empty0 + 8 * s, ((it / TURNS) & 1) ^ 1, &abort_sh,
                                                             p.status));
                        if (!ok) break;
                        float *to = reinterpret_cast<float *>(smem + P::OFF_SCALES) + s * P::SCALES + lane;
#pragma unroll
                        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
                            for (int i = 0; i < EACH; ++i) to[32 * (j * EACH + i)] = x[d][i] * w[d][j];
                        __syncwarp();
                        if (lane < HALVES) mbar_arrive_local(acc_full0 + 8 * (s * HALVES + lane));
                        load(ks + d + AHEAD, x[d], w[d]);
                        ++it;
                    }
            }
        }
        __syncwarp();
    } else {
        if constexpr (P::WIDE) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ------------------------------------------------ drain
        constexpr int GROUPS = P::COLS / 32;             // 32 columns at a time
        const int q = warp & 3, c0 = (warp >> 2) * P::COLS;     // c0: first column of the tile
        const int h = HALVES == 2 ? warp >> 2 : 0;       // the accumulator it drains
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t acc_empty_even = in_even_cta(acc_empty0);
        const float *scales = reinterpret_cast<const float *>(smem + P::OFF_SCALES) +
                              (P::WIDE ? c0 / 128 * 128 + q * 32 + lane : c0);
        // an accumulator has been read
        auto hand_back = [&](int a) {
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_cluster(acc_empty_even + 8 * a);
        };
        uint32_t it = 0;
        F8Iter iter(cut, pair);
        F8Seg sg;
        // the warp acts as one: a lane that saw an abort takes the others along
        while (__all_sync(0xffffffffu, !abort_sh) && iter.next(cut, list, p, sg)) {
            const int row = static_cast<int>(rank) * kHalf + q * 32;     // of this warp, on the M side
            const int n0 = sg.ntile * kTileN;
            const int rows_left = (P::WIDE ? sg.cols : p.N - n0) - row;
            const int cols_left = (P::WIDE ? p.N - n0 : sg.cols) - c0;
            const bool some = rows_left > 0 && cols_left > 0;            // this warp has some of the tile
            const int groups = some ? min(GROUPS, (cols_left + 31) / 32) : 0;
            float acc[GROUPS][32];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[g][i] = 0.0f;
            bool ok = true;
            int left = sg.k1 - sg.k0;
#pragma unroll 1
            for (; left > 0; --left, ++it) {
                const int s = it % TURNS, a = s * HALVES + h;
                ok = __all_sync(0xffffffffu, f8_wait(acc_full0 + 8 * a, (it / TURNS) & 1, &abort_sh, p.status));
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = tmem + lanes + static_cast<uint32_t>(P::ACC_COLS * a + (HALVES == 2 ? 0 : c0));
                if constexpr (P::WIDE) {
                    // (columns past N too: what comes of them is not stored)
                    const float f1 = scales[s * P::SCALES];
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        uint32_t v[32];
                        tmem_ld32(at + 32 * g, v);
                        tmem_wait32(v);
                        if (g == GROUPS - 1) hand_back(a);
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[g][i] = fmaf(__uint_as_float(v[i]), f1, acc[g][i]);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups) {
                            uint32_t v[32];
                            tmem_ld32(at + 32 * g, v);
                            float4 f[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                f[i] = *reinterpret_cast<const float4 *>(scales + s * P::SCALES + 32 * g + 4 * i);
                            tmem_wait32(v);
                            if (g == groups - 1) hand_back(a);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                acc[g][4 * i] = fmaf(__uint_as_float(v[4 * i]), f[i].x, acc[g][4 * i]);
                                acc[g][4 * i + 1] = fmaf(__uint_as_float(v[4 * i + 1]), f[i].y, acc[g][4 * i + 1]);
                                acc[g][4 * i + 2] = fmaf(__uint_as_float(v[4 * i + 2]), f[i].z, acc[g][4 * i + 2]);
                                acc[g][4 * i + 3] = fmaf(__uint_as_float(v[4 * i + 3]), f[i].w, acc[g][4 * i + 3]);
                            }
                        }
                    if (groups == 0) hand_back(a);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_local(sc_empty0 + 8 * s);
            }
            if (!ok) break;                              // a wait ran out
            if (!some) continue;
            if (!sg.whole) {
                // store the part; the warp that comes last adds all parts in order
                auto slot = [&](int pr) {
                    return reinterpret_cast<float2 *>(
                               p.slots + (static_cast<int64_t>(pr) * 4 + (pr == sg.first ? 2 : 0) + rank) * P::SLOT) +
                           static_cast<int64_t>(warp) * GROUPS * 16 * 32 + lane;
                };
                float2 *to = slot(pair);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    if (g < groups)
#pragma unroll
                        for (int i = 0; i < 16; ++i) __stcg(to + (g * 16 + i) * 32, make_float2(acc[g][2 * i], acc[g][2 * i + 1]));
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
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[g][i] = 0.0f;
                for (int pr = sg.first; pr <= sg.last; ++pr) {
                    const float2 *from = slot(pr);
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups)
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 v = __ldcg(from + (g * 16 + i) * 32);
                                acc[g][2 * i] += v.x;
                                acc[g][2 * i + 1] += v.y;
                            }
                }
            }
            if constexpr (P::WIDE) {
                // ---- Y: a lane has a token's columns; 64 bytes of each of the warp's 32 rows at a
                // time go through shared memory, so that four lanes store a row's 64 bytes.  A
                // row's chunk c lies at c ^ (row / 2 % 4): no two of eight rows in one bank.
                unsigned char *turn = smem + P::OFF_OUT + warp * 32 * 64;
                const int esize = p.ytype == 0 ? 4 : 2, piece = 16 / esize;
                unsigned char *y = static_cast<unsigned char *>(p.Y) +
                                   ((static_cast<int64_t>(sg.m0) + row + (lane >> 2)) * p.ldy + n0 + c0 + (lane & 3) * piece) * esize;
                auto turn_out = [&](const uint4 (&u)[4], int col) {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4 *>(turn + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = u[j];
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = r * 8 + (lane >> 2), left = cols_left - col - (lane & 3) * piece;
                        if (at >= rows_left || left <= 0) continue;
                        const uint4 o = *reinterpret_cast<const uint4 *>(turn + at * 64 + (((lane & 3) ^ ((at >> 1) & 3)) << 4));
                        unsigned char *to = y + (static_cast<int64_t>(r) * 8 * p.ldy + col) * esize;
                        if (p.vec && left >= piece) {
                            *reinterpret_cast<uint4 *>(to) = o;
                        } else {
                            const uint32_t h[4] = {o.x, o.y, o.z, o.w};
                            if (esize == 4) {
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    if (j < left) reinterpret_cast<uint32_t *>(to)[j] = h[j];
                            } else {
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (j < left)
                                        reinterpret_cast<uint16_t *>(to)[j] = static_cast<uint16_t>(h[j >> 1] >> (16 * (j & 1)));
                            }
                        }
                    }
                };
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    if (g >= groups) break;
                    uint4 u[4];
                    if (p.ytype == 0) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float *a = acc[g] + 16 * hh + 4 * j;
                                u[j] = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                                                  __float_as_uint(a[3]));
                            }
                            turn_out(u, 32 * g + 16 * hh);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t h[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                h[i] = bf16_pair(acc[g][8 * j + 2 * i], acc[g][8 * j + 2 * i + 1]);
                            }
                            u[j] = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                        turn_out(u, 32 * g);
                    }
                }
            } else {
                // ---- Y: this lane's column n of tokens c0, c0 + 1, ...
                const int n = n0 + row + lane;
                const int64_t first = (static_cast<int64_t>(sg.m0) + c0) * p.ldy;
                if (p.ytype == 1 && p.vec) {
                    // two lanes exchange a value: the even one takes both columns of one token, the
                    // odd one of the next, and a store is 4 bytes
                    const int odd = lane & 1, ne = n - odd;
                    uint16_t *y = static_cast<uint16_t *>(p.Y) + first + odd * p.ldy + ne;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups)
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int c = 32 * g + 2 * i;
                                const float2 v = make_float2(acc[g][2 * i], acc[g][2 * i + 1]);
                                const float got = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.y, 1);
                                const uint32_t both = bf16_pair(odd ? got : v.x, odd ? v.y : got);
                                if (c + odd < cols_left) {
                                    uint16_t *to = y + c * p.ldy;
                                    if (ne + 1 < p.N)
                                        *reinterpret_cast<uint32_t *>(to) = both;
                                    else if (ne < p.N)
                                        *to = static_cast<uint16_t>(both);
                                }
                            }
                } else {
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups)
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 v = make_float2(acc[g][2 * i], acc[g][2 * i + 1]);
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int c = 32 * g + 2 * i + j;
                                    const float u = j ? v.y : v.x;
                                    if (n >= p.N || c >= cols_left) continue;
                                    if (p.ytype == 0)
                                        static_cast<float *>(p.Y)[first + c * p.ldy + n] = u;
                                    else
                                        static_cast<uint16_t *>(p.Y)[first + c * p.ldy + n] = f32_to_bf16_bits(u);
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
        if (P::WIDE && at.numRegs * P::THREADS < 184 * 256 + 72 * 256) return TQ_ERR_DEVICE;
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
    p.nblocks = static_cast<int>((f.N + 127) / 128);
    p.ntiles = static_cast<int>((f.N + kTileN - 1) / kTileN);
    p.Y = f.Y;
    p.ldy = f.ldy;
    p.ytype = f.ytype;
    const int piece = P::WIDE ? 16 : 4;
    p.vec = reinterpret_cast<uintptr_t>(f.Y) % piece == 0 && f.ldy * (f.ytype == 0 ? 4 : 2) % piece == 0 ? 1 : 0;
    p.status = status_word();
    if (!p.status) return TQ_ERR_DEVICE;
    const int most = dev.sms / 2;
    p.counters = static_cast<unsigned int *>(f.ws);
    p.slots = static_cast<unsigned char *>(f.ws) + kF8CounterBytes(most);
    p.min_steps = 2;
    CUtensorMap tmW, tmX;
    if (!make_map_u8(&tmW, f.Wq, p.experts * f.N, f.K, kStepK, P::WIDE ? P::B_BOX : kHalf, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_u8(&tmX, f.Xq, f.M, f.K, kStepK, P::WIDE ? kHalf : P::B_BOX, CU_TENSOR_MAP_SWIZZLE_128B))
        return TQ_ERR_DEVICE;
    // token tiles there may be: one more an expert than whole ones
    const int64_t token_tiles = f.M / NT + (f.M < p.experts ? f.M : p.experts);
    if (token_tiles * p.ntiles > (1ll << 30)) return TQ_ERR_OVERFLOW;
    const int64_t steps = token_tiles * p.ntiles * p.ksteps;
    const int64_t pairs = steps / p.min_steps < 1 ? 1 : (steps / p.min_steps < most ? steps / p.min_steps : most);
    kern<<<static_cast<unsigned>(2 * pairs), P::THREADS, P::smem(p.experts), s>>>(P::WIDE ? tmX : tmW, P::WIDE ? tmW : tmX, p);
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
