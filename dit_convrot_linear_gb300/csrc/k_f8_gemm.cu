// The product of 8-bit floating-point operands with a scale for each block of 128,
//   Y[m][n] = sum_b sx[b][m] * sw[n / 128][b] * sum_{k in block b} xq[m][k] * wq[n][k],
// of one matrix, or of one matrix an expert over rows sorted by expert, on tcgen05
// (kind::f8f6f4: e4m3 operands as they are, at twice the rate of fp16).
//
// A step of K is one scale block, four MMAs of 32.  The accumulator of each step lies
// in TMEM of its own, and the drain warps add it, times its scales, to the sums in
// their registers.  Two forms of a tile:
//   many tokens  128 tokens by 256 columns of Y (128 where that saves a round).  The tokens
//                are the MMA's M side, so that a TMEM lane is a token and a step's scales are
//                one number a thread, acc += (sx[b][token] * sw[block][b]) * part.
//   few tokens   128 columns of Y by up to 64 tokens.  The weights are the M side and the
//                tokens the N side, in steps of 16: an expert's few rows cost no empty rows
//                of a 128-row tile.  The scales differ from column to column and come from
//                shared memory, 4 bytes a lane and value; at 64 tokens that hides behind the
//                weights' stream.
// Warps of a CTA (one an SM):
//   8 drain warps  multiply and add, write Y: a TMEM lane quarter and 128 columns each, or
//                  64 columns, four warps a step in turn, whose sums are put together;
//   MMA warps      one thread of each issues: two a half, that take the steps in turn;
//   copy warp      tensor copies of both operands into the ring (128-byte swizzle);
//   2 scale warps  each step's scales into shared memory, in turn.
//
// What bounds it.  With many tokens a step's MMAs take 512 cycles, and it takes about 950
// (4032 tokens, 4096 to 12288: 185 us, 2200 TFLOP/s).  TMEM holds two steps, so that an
// accumulator comes round every 1900: its MMAs 512, their commit 300, the drain from there
// to the hand-back 390, its arrival 200, and the issue, whose four MMAs and two commits
// hold a thread for 600 (drain and issue by the clock in a build for it; a drain warp waits
// 240 a step, and its sums past the hand-back take 40).  Shared memory is not what binds: a
// step writes and reads 112 KB of it, and one accumulator of 256 columns, with 96 KB, is
// within 3%.  So are the next columns loaded ahead of the sums and 192 registers a drain
// thread.  A step's columns are two accumulators of 128 with MMAs of their own, one filled
// while the other is drained, and four threads issue.  Pairs of CTAs
// (256 x 256, 80 KB a step and CTA) take as long for such a matrix, as the arrivals cross
// to the other SM, and waste more of an expert's last tile: 512 tokens of 64 experts, eight
// each, 2048 x 2048: 87 us against 57; 4096 tokens 178 against 164.  Sixteen drain warps:
// 10% slower.
// Few tokens: the weights' stream, of which an SM draws 42 bytes a ns; six stages of 16 KB
// of it in flight.  In both forms the copies are one thread's, and its instructions a step
// count: a loop over the boxes of the N side in place of two calls costs 10%.
//
// The work is a list of tiles (expert, columns, tokens).  Whole rounds of tiles go to
// the CTAs one by one; the K steps of a last round that would leave CTAs idle are
// shared out evenly.  A CTA that has only part of a tile's steps stores its sums, and
// the warp that comes last at the tile's counter adds all parts in the order of K:
// nobody waits, and the order does not depend on time.  Every wait on an mbarrier is
// bounded: on expiry the CTA records it in the status word, stops, lets what is in
// flight finish (bounded), frees its TMEM and returns.

#include "tq_tc.cuh"

namespace tq {
namespace {

constexpr int kStepK = 128;               // K of a step: one scale block
constexpr int kRowsA = 128;               // rows of the M side a CTA
constexpr int kABytes = kRowsA * kStepK;  // a stage's M side
// Waits for operands are bounded by kF8WaitLimit clock cycles (about 2 s; a build for the
// library's own tests sets TQ_TEST_WAIT_CYCLES), those for what is in flight once one ran
// out by kF8LandLimit each.
#ifdef TQ_TEST_WAIT_CYCLES
constexpr long long kF8WaitLimit = TQ_TEST_WAIT_CYCLES;
#else
constexpr long long kF8WaitLimit = 4000000000ll;
#endif
constexpr long long kF8LandLimit = 250000000ll;
// A build for the library's own tests expects bytes that no copy brings, so that no
// stage completes and the waits run out, with every issued copy landed.
#ifdef TQ_TEST_UNSET_BYTES
constexpr uint32_t kF8Unset = TQ_TEST_UNSET_BYTES;
#else
constexpr uint32_t kF8Unset = 0;
#endif
constexpr unsigned int kStatusF8Timeout = 512u;

template <bool WIDE_>
struct F8Plan {
    static constexpr bool WIDE = WIDE_;                        // many tokens: they are the M side
    static constexpr int TOKENS = WIDE ? 128 : 64;             // of a tile, at most
    static constexpr int YCOLS = WIDE ? 256 : 128;             // weight rows of a tile, at most
    static constexpr int NCOLS = WIDE ? YCOLS : TOKENS;        // the N side
    static constexpr int COLS = WIDE ? 128 : 64;               // of them a drain warp
    static constexpr int SETS = WIDE ? 1 : 2;                  // of drain warps, that take the steps in turn
    static constexpr int DRAIN = 4 * NCOLS / COLS * SETS;      // drain warps
    static constexpr int HALVES = WIDE ? 2 : 1;                // accumulators a step
    static constexpr int ISSUERS = 2 * HALVES, IN_TURN = ISSUERS / HALVES;  // MMA warps; a half's, the steps in turn
    static constexpr int SCALERS = 2;                           // scale warps: the steps in turn
    static constexpr int OTHERS = 8;                           // warps that do not drain
    static constexpr int THREADS = (DRAIN + OTHERS) * 32;
    static constexpr int B_BOX = WIDE ? 128 : 32;               // rows of one tensor copy of the N side
    static constexpr int STAGE = kABytes + NCOLS * kStepK;
    static constexpr int STAGES = WIDE ? 4 : 6;
    static constexpr int TURNS = WIDE ? 2 : 4;                 // steps with accumulators in TMEM
    static constexpr int ACCS = TURNS * HALVES, ACC_COLS = NCOLS / HALVES;
    static constexpr int TMEM = ACC_COLS * ACCS;
    // of a step.  Many tokens: 128 products for each half; few: the tokens', and of the weights
    // the tile's two blocks'
    static constexpr int SCALES = WIDE ? 256 : TOKENS + 4;
    static constexpr int SLOTS = 2 * TURNS;                    // steps with scales in shared memory
    static constexpr int OFF_SCALES = STAGES * STAGE;
    // many tokens: 64 bytes of 32 rows a warp; few: the second set's sums
    static constexpr int OUT_BYTES = WIDE ? DRAIN * 32 * 64 : 4 * 32 * COLS * 4;
    static constexpr int OFF_OUT = OFF_SCALES + SLOTS * SCALES * 4;
    static constexpr int OFF_BARS = OFF_OUT + OUT_BYTES;
    static constexpr int NBARS = 2 * STAGES + 2 * ACCS + 1 + 8;
    static constexpr int OFF_LIST = OFF_BARS + (NBARS * 8 + 15) / 16 * 16;
    // the list of experts: first row, rows, tiles before
    static constexpr int smem(int64_t experts) { return OFF_LIST + static_cast<int>(experts + 1) * 12 + 16; }
    static constexpr int PART = DRAIN * 32 * COLS * 4;         // bytes of a CTA's partial tile
    static constexpr int MIN_STEPS = 4, JOIN_STEPS = WIDE ? 44 : 12;   // of split tiles: steps a CTA, steps saved
    // registers a thread at the launch, then of the drain warps and the others.  Few tokens leave
    // room for a CTA of the next kernel, an operand's quantiser, which then waits where it runs:
    // 16 tokens' layer of 64 experts, eight each, 2048 x 1024, 80 us, and 85 with all registers
    // taken and the list of work made after the wait.
    static constexpr int REGS = WIDE ? 128 : 112, DRAIN_REGS = WIDE ? 176 : 136, OTHER_REGS = WIDE ? 80 : 88;
    static_assert(REGS * THREADS >= 32 * (DRAIN * DRAIN_REGS + OTHERS * OTHER_REGS), "registers");
};
// A wait for a parity tells two neighbouring rounds of a barrier apart, no more: who
// waits for a stage's or an accumulator's round has to have seen the round before it.  So
// those that take the steps in turn meet the same stages and accumulators every time.
template <class P>
constexpr bool f8_turns() {
    return P::STAGES % P::IN_TURN == 0 && P::TURNS % P::IN_TURN == 0 && P::TURNS % P::SETS == 0 && P::TURNS % P::SCALERS == 0;
}
static_assert(f8_turns<F8Plan<true>>() && f8_turns<F8Plan<false>>(), "rounds");
static_assert(F8Plan<true>::smem(TQ_MAX_EXPERTS) <= 226 * 1024 && F8Plan<false>::smem(TQ_MAX_EXPERTS) <= 226 * 1024,
              "shared memory");

constexpr int kF8MaxDrain = 8, kF8MaxParts = 4, kF8MinRows = 32;

struct F8Params {
    const float *sx;
    int64_t M;
    const int32_t *offsets;
    int experts;
    const float *sw;
    int N, ksteps, nblocks, ntiles;      // nblocks: scale blocks of N; ntiles: tiles of N
    int ycols;                           // weight rows of a tile (few tokens: at most 128, even)
    void *Y;
    int64_t ldy;
    int ytype, vec;                      // vec: rows of Y allow stores of 16 bytes, 4 or 2
    unsigned int *status;
    unsigned int *counters;              // [CTAs][kF8MaxDrain]
    unsigned char *parts;                // [CTAs][2][PART]
};

// A piece of work: the tile's place, K steps k0 .. k1 - 1, and for a piece of a
// split tile the CTAs that have its first and last step.
struct F8Seg {
    int e, ntile, m0, cols, k0, k1;      // cols: tokens of the tile
    bool whole;
    int first, last;
};

// The list of work, in shared memory: of each expert its first row, its rows and the
// token tiles before it (one more entry), and how the tiles are cut.
struct F8Cut {
    int whole;       // tiles computed whole
    int units;       // K steps of the others,
    int use;         // shared by this many CTAs
};

// The pieces of work of a CTA, in order.  (What does not change lies in shared
// memory: the drain warps have few registers to spare.)
struct F8Iter {
    int i, u0;
    __device__ explicit F8Iter(const F8Cut &c)
        : i(0), u0(static_cast<int>(blockIdx.x) < c.use ? bound(c, blockIdx.x) : 0) {}
    static __device__ int bound(const F8Cut &c, int q) {
        return static_cast<int>(static_cast<long long>(c.units) * q / c.use);
    }
    // the CTA whose steps include x
    static __device__ int owner(const F8Cut &c, int x) {
        int q = static_cast<int>(static_cast<long long>(x) * c.use / c.units);
        while (q + 1 < c.use && bound(c, q + 1) <= x) ++q;
        while (q > 0 && bound(c, q) > x) --q;
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
        const int cta = blockIdx.x, ksteps = p.ksteps;
        const int t = cta + i * static_cast<int>(gridDim.x);
        if (t < c.whole) {
            ++i;
            place(list, p, t, s);
            s.k0 = 0;
            s.k1 = ksteps;
            s.whole = true;
            return true;
        }
        const int u1 = cta < c.use ? bound(c, cta + 1) : 0;
        if (u0 >= u1) return false;
        const int tl = u0 / ksteps, ts = tl * ksteps;
        place(list, p, c.whole + tl, s);
        s.k0 = u0 - ts;
        s.k1 = min(u1, ts + ksteps) - ts;
        s.whole = s.k0 == 0 && s.k1 == ksteps;
        s.first = s.last = cta;
        if (!s.whole) {
            s.first = owner(c, ts);
            s.last = owner(c, ts + ksteps - 1);
        }
        u0 = ts + s.k1;
        return true;
    }
};

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

// A warp's wait: all or none of its lanes go on.
__device__ __forceinline__ bool f8_wait_warp(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *status) {
    const bool ok = f8_wait(bar, parity, abort, status);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void f8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u));
}
__device__ __forceinline__ void f8_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void f8_prefetch(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}

// A place in a ring of N stages and the parity of the round that fills it.
template <int N>
struct F8Ring {
    int s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void on(int n) {
        s += n;
        if (s >= N) {
            s -= N;
            round ^= 1u;
        }
    }
};

// K-major operand of 128-byte rows in the 128-byte swizzle: groups of eight rows
// 1024 bytes apart; 32 values on along K are 32 bytes on.
__device__ __forceinline__ uint64_t f8_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Columns of this lane's row, read and waited for.
__device__ __forceinline__ void tmem_read16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_read32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <class P>
__global__ void __maxnreg__(P::REGS)
k_linear_f8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const F8Params p) {
    constexpr int DRAIN = P::DRAIN, STAGES = P::STAGES, ACCS = P::ACCS, TURNS = P::TURNS, HALVES = P::HALVES;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + P::OFF_BARS);
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_sh;
    __shared__ F8Cut cut;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
    const uint32_t acc_full0 = empty0 + 8 * STAGES, acc_empty0 = acc_full0 + 8 * ACCS;
    const uint32_t done = acc_empty0 + 8 * ACCS, sum_full0 = done + 8, sum_empty0 = sum_full0 + 32;

    if (threadIdx.x == 32) {
        auto init = [](uint32_t bar, uint32_t n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n));
        };
        for (int s = 0; s < STAGES; ++s) {
            init(full0 + 8 * s, 1);
            init(empty0 + 8 * s, HALVES);
        }
        for (int a = 0; a < ACCS; ++a) {
            init(acc_full0 + 8 * a, 2);             // the step's MMAs, and its scales
            init(acc_empty0 + 8 * a, DRAIN / HALVES / P::SETS);
        }
        for (int i = 0; i < 8; ++i) init(sum_full0 + 8 * i, 1);         // a quarter's sums: put there, taken
        init(done, P::ISSUERS);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_sh = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
    }
    // What an earlier kernel wrote is read, and the workspace used, after pdl_wait; the TMEM
    // is taken then too (that kernel's CTAs may still need theirs), and the next kernel may
    // start once this one has its own.  The list of work is made before, from offsets that may
    // still change (it is made again if they did), and the first weights come into L2 (coherent:
    // whoever writes them still may).
    const int *list = reinterpret_cast<const int *>(smem + P::OFF_LIST);
    int *row0 = reinterpret_cast<int *>(smem + P::OFF_LIST), *rows = row0 + p.experts + 1, *tiles = rows + p.experts + 1;
    const volatile int32_t *offsets = p.offsets;
    bool bad = false;
    auto make_list = [&]() {
        int total = static_cast<int>((p.M + P::TOKENS - 1) / P::TOKENS);       // token tiles
        if (p.offsets == nullptr) {
            if (lane == 0) {
                row0[0] = 0;
                rows[0] = static_cast<int>(p.M);
                tiles[0] = 0;
                tiles[1] = total;
            }
        } else {
            // an expert whose range is out of order has no rows
            int sum = 0, most = INT32_MIN;
            bad = false;
            for (int e0 = 0; e0 < p.experts; e0 += 32) {
                const int e = e0 + lane;
                const bool in = e < p.experts;
                const int a = in ? row0[e] : INT32_MIN, b = in ? row0[e + 1] : INT32_MIN;
                int top = a;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, top, o);
                    if (lane >= o) top = max(top, v);
                }
                top = max(top, most);               // the largest offset so far
                const bool ok = a >= 0 && b >= a && b <= p.M && a >= top;
                const int n = in && ok ? b - a : 0;
                bad |= in && !ok;
                const int t = (n + P::TOKENS - 1) / P::TOKENS;
                int s = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, s, o);
                    if (lane >= o) s += v;
                }
                if (in) {
                    rows[e] = n;
                    tiles[e] = sum + s - t;
                }
                sum += __shfl_sync(0xffffffffu, s, 31);
                most = __shfl_sync(0xffffffffu, top, 31);
            }
            if (lane == 0) tiles[p.experts] = sum;
            total = sum;
        }
        if (lane == 0) {
            // The tiles of a last round that leaves CTAs idle are split where that saves more
            // steps than the joining costs, among at most kF8MaxParts CTAs a tile (a tile whose ends
            // lie within two CTAs' shares has a part more).  (Many tokens, 4096
            // to 12288: 512 of them, whose last 40 tiles of 32 steps could be of 9, 38 us whole and
            // 50 split.  12288 to 4096: 4032, the last 56 tiles of 96 steps in parts of 35, 199
            // us whole and 188 split.)
            const int n = total * p.ntiles, ctas = gridDim.x, rest = n % ctas;
            const int units = rest * p.ksteps;
            const int use = max(1, min(min(ctas, rest * kF8MaxParts), units / P::MIN_STEPS));
            const bool split = rest > 0 && p.ksteps - (units + use - 1) / use >= P::JOIN_STEPS;
            cut.whole = split ? n - rest : n;
            cut.units = split ? units : 0;
            cut.use = use;
        }
    };
    if (p.offsets) {
        for (int e = threadIdx.x; e <= p.experts; e += P::THREADS) row0[e] = offsets[e];
        __syncthreads();
    }
    if (warp == 0) make_list();
    __syncthreads();
    // weight rows of a tile, and columns of its accumulator h: tokens, or weight rows, rounded
    // up to 16 (one without any still takes part, and nothing of it is stored)
    auto tile_rows = [&](const F8Seg &sg) { return min(p.ycols, p.N - sg.ntile * p.ycols); };
    auto mma_n = [&](const F8Seg &sg, int h) {
        const int n = P::WIDE ? min(P::ACC_COLS, tile_rows(sg) - h * P::ACC_COLS) : sg.cols;
        return (max(n, 1) + 15) / 16 * 16;
    };
    // The copy warp's work on a tile: where its operands lie, and a step's copies into the
    // stage s, the weights (with the bytes that are expected there) and the tokens.  The N side
    // comes in one box or two, as many as hold the tile's columns.
    struct Source {
        int wrow, xrow, boxes;
        uint32_t bytes;
    };
    auto source = [&](const F8Seg &sg) {
        Source c;
        c.boxes = ((P::WIDE ? tile_rows(sg) : sg.cols) + P::B_BOX - 1) / P::B_BOX;
        c.bytes = (c.boxes * P::B_BOX + (P::WIDE ? kRowsA : p.ycols)) * kStepK + kF8Unset;
        c.wrow = sg.e * p.N + sg.ntile * p.ycols;
        c.xrow = sg.m0;
        return c;
    };
    const uint32_t stage0 = smem_u32(smem);
    auto copy_a = [&](int s, int k, int row) { tma_load_2d(stage0 + s * P::STAGE, &tmA, k, row, full0 + 8 * s); };
    auto copy_b = [&](int boxes, int s, int k, int row) {
        const uint32_t at = stage0 + s * P::STAGE + kABytes;
        tma_load_2d(at, &tmB, k, row, full0 + 8 * s);
        if (boxes > 1) tma_load_2d(at + P::B_BOX * kStepK, &tmB, k, row + P::B_BOX, full0 + 8 * s);
    };
    auto copy_weights = [&](const Source &c, int s, int k) {
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full0 + 8 * s), "r"(c.bytes) : "memory");
        if constexpr (P::WIDE) copy_b(c.boxes, s, k, c.wrow);
        else copy_a(s, k, c.wrow);
    };
    auto copy_tokens = [&](const Source &c, int s, int k) {
        if constexpr (P::WIDE) copy_a(s, k, c.xrow);
        else copy_b(c.boxes, s, k, c.xrow);
    };
    if (warp == DRAIN + P::ISSUERS && lane == 0) {
        F8Iter iter(cut);
        F8Seg sg;
        if (iter.next(cut, list, p, sg)) {
            const Source c = source(sg);
            for (int k = sg.k0; k < min(sg.k1, sg.k0 + STAGES); ++k) {
                f8_prefetch(P::WIDE ? &tmB : &tmA, k * kStepK, c.wrow);
                if (P::WIDE && c.boxes > 1) f8_prefetch(&tmB, k * kStepK, c.wrow + P::B_BOX);
            }
        }
    }
    __syncwarp();
    pdl_wait();
    if (p.offsets) {
        int changed = 0;
        for (int e = threadIdx.x; e <= p.experts; e += P::THREADS) {
            const int32_t now = offsets[e];
            if (now != row0[e]) {            // (the prefetch above does not read it)
                row0[e] = now;
                changed = 1;
            }
        }
        if (__syncthreads_or(changed)) {
            if (warp == 0) make_list();
            __syncthreads();
        }
        if (bad) atomicOr(p.status, kStatusIndex);
    }
    if (warp == DRAIN) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_base_sh)), "r"(static_cast<uint32_t>(P::TMEM)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_base_sh;
    pdl_launch_dependents();

    if (warp >= DRAIN) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::OTHER_REGS));
        if (warp < DRAIN + P::ISSUERS) {
            // -------------------------------------------- MMA issue (one thread a warp)
            if (lane == 0) {
                const int h = (warp - DRAIN) % HALVES;
                const uint32_t turn = (warp - DRAIN) / HALVES;
                uint32_t it = 0, mine = turn;            // mine: the next step of this thread's
                F8Ring<STAGES> at;
                at.on(turn);
                F8Iter iter(cut);
                F8Seg sg;
                while (!abort_sh && iter.next(cut, list, p, sg)) {
                    // D fp32, A and B e4m3, K-major, M = 128
                    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(mma_n(sg, h) >> 3) << 17) | (8u << 24);
                    const uint32_t end = it + sg.k1 - sg.k0;
                    for (; mine < end; mine += P::IN_TURN, at.on(P::IN_TURN)) {
                        const int a = (mine % TURNS) * HALVES + h;
                        if (!f8_wait(full0 + 8 * at.s, at.round, &abort_sh, p.status)) break;
                        if (!f8_wait(acc_empty0 + 8 * a, ((mine / TURNS) & 1) ^ 1, &abort_sh, p.status)) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t d = tmem + static_cast<uint32_t>(P::ACC_COLS * a);
                        const uint64_t ad = f8_desc(stage0 + at.s * P::STAGE);
                        const uint64_t bd = f8_desc(stage0 + at.s * P::STAGE + kABytes + h * P::ACC_COLS * kStepK);
#pragma unroll
                        for (int kk = 0; kk < kStepK / 32; ++kk) f8_mma(d, ad + 2 * kk, bd + 2 * kk, idesc, kk > 0);
                        f8_commit(acc_full0 + 8 * a);
                        f8_commit(empty0 + 8 * at.s);
                    }
                    it = end;
                }
                // let every issued MMA finish before the TMEM is released
                f8_commit(done);
                const long long t0 = clock64();
                while (!f8_try(done, 0) && clock64() - t0 < kF8LandLimit) {
                }
            }
        } else if (warp == DRAIN + P::ISSUERS) {
            // -------------------------------------------- tensor copies
            if (lane == 0) {
                uint32_t it = 0;
                F8Ring<STAGES> at;
                F8Iter iter(cut);
                F8Seg sg;
                while (!abort_sh && iter.next(cut, list, p, sg)) {
                    const Source c = source(sg);
                    for (int k = sg.k0 * kStepK; k < sg.k1 * kStepK; k += kStepK, ++it, at.on(1)) {
                        if (!f8_wait(empty0 + 8 * at.s, at.round ^ 1u, &abort_sh, p.status)) break;
                        copy_weights(c, at.s, k);
                        copy_tokens(c, at.s, k);
                    }
                }
                // after a wait ran out: the copies in flight land before the CTA leaves
                if (abort_sh)
                    for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j) {
                        const long long t0 = clock64();
                        while (!f8_try(full0 + 8 * (j % STAGES), (j / STAGES) & 1) &&
                               clock64() - t0 < kF8LandLimit) {
                        }
                    }
            }
        } else if (warp < DRAIN + P::ISSUERS + 1 + P::SCALERS) {
            // -------------------------------------------- scales
            // Each step's sx * sw into its slot, loaded AHEAD steps before.  Many tokens: this CTA's
            // tokens with the first scale block of columns, then with the second.  Few: sx of each
            // token, and sw of the tile's first block of weight rows and the next.  (Places past the
            // tile's rows or N take their last one's; what comes of them is not stored.)  A slot is
            // free again 2 * TURNS steps later: step it - TURNS has its sums only after step
            // it - 2 * TURNS was drained.
            constexpr int SC = P::SCALERS, AHEAD = 2, EACH = P::WIDE ? 4 : P::TOKENS / 32;
            const int turn = warp - (DRAIN + P::ISSUERS + 1);
            uint32_t it = 0;
            F8Iter iter(cut);
            F8Seg sg;
            while (__all_sync(0xffffffffu, !abort_sh) && iter.next(cut, list, p, sg)) {
                const int skip = (turn + SC - static_cast<int>(it % SC)) % SC;      // steps until this warp's first
                int off[EACH];
#pragma unroll
                for (int i = 0; i < EACH; ++i) off[i] = min(lane + 32 * i, sg.cols - 1);
                const int nb = sg.ntile * p.ycols / 128;
                const float *sx = p.sx + (sg.k0 + skip) * p.M + sg.m0;
                const float *sw = p.sw + (static_cast<int64_t>(sg.e) * p.nblocks + nb) * p.ksteps + sg.k0 + skip;
                const int second = nb + 1 < p.nblocks ? p.ksteps : 0;    // the second block's scales, from the first's
                float x[AHEAD][EACH], w[AHEAD][2];
                int left = sg.k1 - sg.k0 - skip;                         // steps to the piece's end, from the next load
                auto load = [&](float (&xs)[EACH], float (&ws)[2]) {
                    if (left > 0) {
#pragma unroll
                        for (int i = 0; i < EACH; ++i) xs[i] = __ldg(sx + off[i]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) ws[j] = __ldg(sw + j * second);
                    }
                    sx += SC * p.M;
                    sw += SC;
                    left -= SC;
                };
#pragma unroll
                for (int d = 0; d < AHEAD; ++d) load(x[d], w[d]);
                bool ok = true;
                uint32_t j = it + skip;
                it += sg.k1 - sg.k0;
                while (ok && j < it)
#pragma unroll
                    for (int d = 0; d < AHEAD; ++d) {
                        if (!ok || j >= it) break;
                        const int s = j % TURNS;
                        if (j >= TURNS)
#pragma unroll
                            for (int h = 0; h < HALVES; ++h)
                                ok = ok && f8_wait_warp(acc_full0 + 8 * (s * HALVES + h), (j / TURNS - 1) & 1, &abort_sh, p.status);
                        if (!ok) break;
                        float *to = reinterpret_cast<float *>(smem + P::OFF_SCALES) + j % P::SLOTS * P::SCALES + lane;
                        if constexpr (P::WIDE) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int i = 0; i < EACH; ++i) to[32 * (h * EACH + i)] = x[d][i] * w[d][h];
                        } else {
#pragma unroll
                            for (int i = 0; i < EACH; ++i) to[32 * i] = x[d][i];
                            if (lane < 2) to[P::TOKENS] = lane == 0 ? w[d][0] : w[d][1];
                        }
                        __syncwarp();
                        if (lane < HALVES) mbar_arrive_local(acc_full0 + 8 * (s * HALVES + lane));
                        load(x[d], w[d]);
                        j += SC;
                    }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::DRAIN_REGS));
        // ------------------------------------------------ drain
        constexpr int GROUPS = P::COLS / 16;             // 16 columns at a time
        const int q = warp & 3, c0 = P::WIDE ? (warp >> 2) * P::COLS : 0;     // c0: first column of the tile
        const uint32_t set = P::SETS == 2 ? warp >> 2 : 0;
        uint32_t sums = 0;                               // tiles whose sums the sets have put together
        const int h = c0 / P::ACC_COLS;                  // the accumulator it drains
        const uint32_t lanes = (static_cast<uint32_t>(q * 32) << 16) + c0 % P::ACC_COLS;
        const float *scales = reinterpret_cast<const float *>(smem + P::OFF_SCALES) +
                              (P::WIDE ? c0 / 128 * 128 + q * 32 + lane : c0);
        // an accumulator has been read
        auto hand_back = [&](int a) {
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive_local(acc_empty0 + 8 * a);
        };
        uint32_t it = 0;
        F8Iter iter(cut);
        F8Seg sg;
        // the warp acts as one: a lane that saw an abort takes the others along
        while (__all_sync(0xffffffffu, !abort_sh) && iter.next(cut, list, p, sg)) {
            const int n0 = sg.ntile * p.ycols, row = q * 32;      // row: of this warp, on the M side
            static_assert(!P::WIDE || P::SCALES == P::NCOLS, "a scale a token and half");
            const int rows_left = (P::WIDE ? sg.cols : tile_rows(sg)) - row;
            const int block = P::TOKENS + (n0 + row + lane) / 128 - n0 / 128;   // few tokens: where this lane's sw is
            const int cols_left = (P::WIDE ? tile_rows(sg) : sg.cols) - c0;
            const bool some = rows_left > 0 && cols_left > 0;            // this warp has some of the tile
            const int groups = some ? min(GROUPS, (cols_left + 15) / 16) : 0;
            float acc[GROUPS][16];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[g][i] = 0.0f;
            bool ok = true;
            int left = sg.k1 - sg.k0;
#pragma unroll 1
            for (; left > 0; --left, ++it) {
                if (P::SETS == 2 && (it & 1) != set) continue;
                const int s = it % TURNS, a = s * HALVES + h;
                ok = f8_wait_warp(acc_full0 + 8 * a, (it / TURNS) & 1, &abort_sh, p.status);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = tmem + lanes + static_cast<uint32_t>(P::ACC_COLS * a);
                const float *f = scales + it % P::SLOTS * P::SCALES;
                if constexpr (P::WIDE) {
                    // (columns past N too: what comes of them is not stored)
                    const float f1 = *f;
#pragma unroll
                    for (int g = 0; g < GROUPS; g += 2) {
                        uint32_t v[32];
                        tmem_read32(at + 16 * g, v);
                        if (g == GROUPS - 2) {
                            hand_back(a);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            acc[g + i / 16][i % 16] = fmaf(__uint_as_float(v[i]), f1, acc[g + i / 16][i % 16]);
                    }
                } else {
                    const float w = f[block];
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups) {
                            float4 x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(f + 16 * g + 4 * i);
                            uint32_t v[16];
                            tmem_read16(at + 16 * g, v);
                            if (g == groups - 1) hand_back(a);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                x[i].x *= w;
                                x[i].y *= w;
                                x[i].z *= w;
                                x[i].w *= w;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                acc[g][4 * i] = fmaf(__uint_as_float(v[4 * i]), x[i].x, acc[g][4 * i]);
                                acc[g][4 * i + 1] = fmaf(__uint_as_float(v[4 * i + 1]), x[i].y, acc[g][4 * i + 1]);
                                acc[g][4 * i + 2] = fmaf(__uint_as_float(v[4 * i + 2]), x[i].z, acc[g][4 * i + 2]);
                                acc[g][4 * i + 3] = fmaf(__uint_as_float(v[4 * i + 3]), x[i].w, acc[g][4 * i + 3]);
                            }
                        }
                    if (groups == 0) hand_back(a);
                }
            }
            if (!ok) break;                              // a wait ran out
            if (!some) continue;
            if constexpr (P::SETS == 2) {
                // the first set's warp of the same quarter takes the second's sums and goes on
                float *put = reinterpret_cast<float *>(smem + P::OFF_OUT) + q * P::COLS * 32 + lane;
                const uint32_t mine = sums++;
                if (set == 1) {
                    if (!f8_wait_warp(sum_empty0 + 8 * q, (mine & 1) ^ 1, &abort_sh, p.status)) break;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups)
#pragma unroll
                            for (int i = 0; i < 16; ++i) put[(16 * g + i) * 32] = acc[g][i];
                    __syncwarp();
                    if (lane == 0) mbar_arrive_local(sum_full0 + 8 * q);
                    continue;
                }
                if (!f8_wait_warp(sum_full0 + 8 * q, mine & 1, &abort_sh, p.status)) break;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    if (g < groups)
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[g][i] += put[(16 * g + i) * 32];
                __syncwarp();
                if (lane == 0) mbar_arrive_local(sum_empty0 + 8 * q);
            }
            // ---- Y of many tokens: a lane has 32 columns of a token.  64 bytes of each of the
            // warp's 32 rows at a time go through shared memory, so that four lanes store a row's 64
            // bytes (16 or 32 lanes where Y's rows are not aligned to 16: 3974 tokens of 272 to 1730,
            // bf16, 16.5 us, and 42 with 16 bytes a lane in pieces; to 1728 12.3).  A row's chunk c lies at
            // c ^ (row / 2 % 4): no two of eight rows in one bank.
            unsigned char *turn = smem + P::OFF_OUT + warp * 32 * 64;
            const int esize = p.ytype == 0 ? 4 : 2, piece = 16 / esize;
            unsigned char *y = static_cast<unsigned char *>(p.Y) +
                               ((static_cast<int64_t>(sg.m0) + row) * p.ldy + n0 + c0) * esize;
            unsigned char *y16 = y + (static_cast<int64_t>(lane >> 2) * p.ldy + (lane & 3) * piece) * esize;
            auto turn_out = [&](const uint4 (&u)[4], int col) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4 *>(turn + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = u[j];
                __syncwarp();
                if (p.vec == 16) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = r * 8 + (lane >> 2), left = cols_left - col - (lane & 3) * piece;
                        if (at >= rows_left || left <= 0) continue;
                        const uint4 o = *reinterpret_cast<const uint4 *>(turn + at * 64 + (((lane & 3) ^ ((at >> 1) & 3)) << 4));
                        unsigned char *to = y16 + (static_cast<int64_t>(r) * 8 * p.ldy + col) * esize;
                        if (left >= piece) {
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
                } else if (p.vec == 4) {
                    // 4 bytes a lane, 16 lanes a row
                    const int w = lane & 15, c = col + w * 4 / esize;
#pragma unroll 4
                    for (int r = 0; r < 16; ++r) {
                        const int at = r * 2 + (lane >> 4);
                        if (at >= rows_left || c >= cols_left) continue;
                        const uint32_t o = *reinterpret_cast<const uint32_t *>(
                            turn + at * 64 + (((w >> 2) ^ ((at >> 1) & 3)) << 4) + (w & 3) * 4);
                        unsigned char *to = y + (static_cast<int64_t>(at) * p.ldy + c) * esize;
                        if (esize == 4 || c + 1 < cols_left)
                            *reinterpret_cast<uint32_t *>(to) = o;
                        else
                            *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(o);
                    }
                } else {
                    // (rows of bf16 that begin between words) a value a lane
#pragma unroll 4
                    for (int at = 0; at < 32; ++at) {
                        if (at >= rows_left || col + lane >= cols_left) continue;
                        reinterpret_cast<uint16_t *>(y)[static_cast<int64_t>(at) * p.ldy + col + lane] =
                            *reinterpret_cast<const uint16_t *>(
                                turn + at * 64 + (((lane >> 3) ^ ((at >> 1) & 3)) << 4) + (lane & 7) * 2);
                    }
                }
            };
            auto store = [&](const float (&x0)[16], const float (&x1)[16], int col) {
                uint4 u[4];
                if (p.ytype == 0) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float *x = half ? x1 : x0;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            u[j] = make_uint4(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                                              __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]));
                        turn_out(u, col + 16 * half);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float *x = (j < 2 ? x0 : x1) + 8 * (j & 1);
                        u[j] = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]),
                                          bf16_pair(x[6], x[7]));
                    }
                    turn_out(u, col);
                }
            };
            if (!sg.whole) {
                // store the part; the warp that comes last adds all parts in order
                auto part = [&](int cta) {
                    return reinterpret_cast<float2 *>(
                               p.parts + (static_cast<int64_t>(cta) * 2 + (cta == sg.first ? 1 : 0)) * P::PART) +
                           static_cast<int64_t>(warp) * GROUPS * 8 * 32 + lane;
                };
                float2 *to = part(blockIdx.x);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    if (g < groups)
#pragma unroll
                        for (int i = 0; i < 8; ++i) __stcg(to + (g * 8 + i) * 32, make_float2(acc[g][2 * i], acc[g][2 * i + 1]));
                __threadfence();
                __syncwarp();
                unsigned int *counter = p.counters + sg.first * kF8MaxDrain + warp;
                unsigned int before = 0;
                if (lane == 0) before = atomicAdd(counter, 1u);
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before != static_cast<unsigned int>(sg.last - sg.first)) continue;
                __threadfence();
                if (lane == 0) *counter = 0u;
                // (what bounds the join is its trips to memory: as many columns and parts at a
                // time as there are registers for)
                constexpr int PARTS = P::WIDE ? 3 : 2, CHUNK = P::WIDE ? 2 : 1;
#pragma unroll
                for (int g = 0; g < GROUPS; g += CHUNK) {
                    if (g >= groups) break;
                    float sum[CHUNK][16];
#pragma unroll
                    for (int i = 0; i < CHUNK * 16; ++i) sum[i / 16][i % 16] = 0.0f;
                    for (int p0 = sg.first; p0 <= sg.last; p0 += PARTS) {
                        float2 v[PARTS][CHUNK * 8];
#pragma unroll
                        for (int j = 0; j < PARTS; ++j) {
                            const float2 *from = part(min(p0 + j, sg.last)) + g * 8 * 32;
#pragma unroll
                            for (int i = 0; i < CHUNK * 8; ++i) v[j][i] = __ldcg(from + i * 32);
                        }
#pragma unroll
                        for (int j = 0; j < PARTS; ++j)
                            if (p0 + j <= sg.last)
#pragma unroll
                                for (int i = 0; i < CHUNK * 8; ++i) {
                                    sum[i / 8][i % 8 * 2] += v[j][i].x;
                                    sum[i / 8][i % 8 * 2 + 1] += v[j][i].y;
                                }
                    }
                    if constexpr (P::WIDE) {
                        store(sum[0], sum[CHUNK - 1], 16 * g);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[g][i] = sum[0][i];
                    }
                }
                if (P::WIDE) continue;
            }
            if constexpr (P::WIDE) {
#pragma unroll
                for (int g = 0; g < GROUPS; g += 2)
                    if (g < groups) store(acc[g], acc[g + 1], 16 * g);
            } else {
                // ---- Y: this lane's column n of tokens c0, c0 + 1, ...
                const int n = n0 + row + lane, n_end = min(p.N, n0 + p.ycols);
                const int64_t first = (static_cast<int64_t>(sg.m0) + c0) * p.ldy;
                if (p.ytype == 1 && p.vec >= 4) {
                    // two lanes exchange a value: the even one takes both columns of one token, the
                    // odd one of the next, and a store is 4 bytes
                    const int odd = lane & 1, ne = n - odd;
                    uint16_t *y = static_cast<uint16_t *>(p.Y) + first + odd * p.ldy + ne;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int c = 16 * g + 2 * i;
                                const float2 v = make_float2(acc[g][2 * i], acc[g][2 * i + 1]);
                                const float got = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.y, 1);
                                const uint32_t both = bf16_pair(odd ? got : v.x, odd ? v.y : got);
                                if (c + odd < cols_left) {
                                    uint16_t *to = y + c * p.ldy;
                                    if (ne + 1 < n_end)
                                        *reinterpret_cast<uint32_t *>(to) = both;
                                    else if (ne < n_end)
                                        *to = static_cast<uint16_t>(both);
                                }
                            }
                } else {
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        if (g < groups)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 v = make_float2(acc[g][2 * i], acc[g][2 * i + 1]);
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int c = 16 * g + 2 * i + j;
                                    const float u = j ? v.y : v.x;
                                    if (n >= n_end || c >= cols_left) continue;
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
    // (The MMAs in flight have ended: their issuers waited for them above.)
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == DRAIN) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(P::TMEM)));
    }
}

constexpr size_t f8_counter_bytes(int ctas) {
    return (static_cast<size_t>(ctas) * kF8MaxDrain * 4 + 255) / 256 * 256;
}

template <bool WIDE>
tq_status launch_f8(const F8Product &f, int ycols, const DeviceInfo &dev, cudaStream_t s) {
    using P = F8Plan<WIDE>;
    auto kern = k_linear_f8<P>;
    if (dev.id < 0 || dev.id >= 64 || dev.sms < 1) return TQ_ERR_DEVICE;
    static bool configured[64] = {false};
    if (!configured[dev.id]) {
        cudaFuncAttributes at;
        cudaError_t e = cudaFuncGetAttributes(&at, kern);
        if (e != cudaSuccess) return cuda_fail(e);
        // the warps' own register counts have to be covered by the launch's
        if (at.numRegs * P::THREADS < 32 * (P::DRAIN * P::DRAIN_REGS + P::OTHERS * P::OTHER_REGS))
            return TQ_ERR_DEVICE;
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
    p.ycols = ycols;
    if (!WIDE && !f.offsets) {
        // Few tokens of one matrix: tiles of 128 rows, the steps of the last round split, or tiles
        // of fewer rows, as many as CTAs.  A step of r rows takes about 3 r ns (what an SM draws
        // from the DRAM) and 250 at least; joining takes 5 us, a round of smaller tiles 1.5 more
        // to begin.  48 tokens of 12288 x 4096: 96 tiles 18 us, 150 of 82 rows 17; 64 of 4096 x
        // 12288: 128 tiles of 32 rows 42, 32 in four parts 22.  (The device splits tiles of fewer
        // rows too, by JOIN_STEPS, which this estimate leaves out: it does at 16 to 22 steps.
        // 64 to 512 rows of 2048: one and 16 tokens 7.0 to 7.5 us split, 7.5 to 8.1 whole; 64
        // tokens 11.0 to 12.7 and 10.8 to 11.1.)
        const int64_t by_tokens = (f.M + P::TOKENS - 1) / P::TOKENS, sms = dev.sms;
        auto whole = [&](int64_t rows) {
            const int64_t tiles = by_tokens * ((f.N + rows - 1) / rows);
            return (tiles + sms - 1) / sms * p.ksteps * (3 * rows > 250 ? 3 * rows : 250);
        };
        const int64_t tiles = by_tokens * ((f.N + 127) / 128);
        const int64_t parts = tiles < sms ? (sms / tiles < kF8MaxParts ? sms / tiles : kF8MaxParts) : 1;
        int64_t large = whole(128);
        if (parts > 1 && p.ksteps - p.ksteps / parts >= P::JOIN_STEPS && large / parts + 5000 < large)
            large = large / parts + 5000;
        const int64_t most = (tiles + sms - 1) / sms * sms / by_tokens, even = ((f.N + most - 1) / most + 1) / 2 * 2;
        const int64_t rows = even < kF8MinRows ? kF8MinRows : even;
        if (rows < 128 && whole(rows) + 1500 < large) p.ycols = static_cast<int>(rows);
    }
    p.ntiles = static_cast<int>((f.N + p.ycols - 1) / p.ycols);
    p.Y = f.Y;
    p.ldy = f.ldy;
    p.ytype = f.ytype;
    const uint64_t step = reinterpret_cast<uintptr_t>(f.Y) | static_cast<uint64_t>(f.ldy * (f.ytype == 0 ? 4 : 2));
    p.vec = step % 16 == 0 ? 16 : (step % 4 == 0 ? 4 : 2);
    p.status = status_word();
    if (!p.status) return TQ_ERR_DEVICE;
    p.counters = static_cast<unsigned int *>(f.ws);
    p.parts = static_cast<unsigned char *>(f.ws) + f8_counter_bytes(dev.sms);
    CUtensorMap tmW, tmX;
    if (!make_map_u8(&tmW, f.Wq, p.experts * f.N, f.K, kStepK, WIDE ? P::B_BOX : p.ycols, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_u8(&tmX, f.Xq, f.M, f.K, kStepK, WIDE ? kRowsA : P::B_BOX, CU_TENSOR_MAP_SWIZZLE_128B))
        return TQ_ERR_DEVICE;
    // token tiles there may be: one more an expert than whole ones
    const int64_t token_tiles = f.M / P::TOKENS + (f.M < p.experts ? f.M : p.experts);
    if (token_tiles * p.ntiles > (1ll << 30)) return TQ_ERR_OVERFLOW;
    const int64_t tiles = token_tiles * p.ntiles, parts = p.ksteps / P::MIN_STEPS;
    const int64_t pieces = tiles * (parts < 1 ? 1 : (parts < kF8MaxParts ? parts : kF8MaxParts));
    const int64_t ctas = pieces < 1 ? 1 : (pieces < dev.sms ? pieces : dev.sms);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(P::THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(P::smem(p.experts));
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, WIDE ? tmX : tmW, WIDE ? tmW : tmX, p);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace

// counters, then two parts of a tile a CTA
size_t f8_workspace_bytes(const DeviceInfo &dev) {
    return f8_counter_bytes(dev.sms) + static_cast<size_t>(dev.sms) * 2 * F8Plan<true>::PART;
}

// The form that takes the least time by rounds of tiles and the time of a step in 10 ns,
// with rows spread evenly over the experts; the weights of a lone tile come from the DRAM.
// Measured with 4096 to 12288: 48 tokens 16.6 us (few) and 19.9 (many, 128 columns); 65:
// 33.7, 19.6 and with 256 columns 21.5; 256: 49, 34.5 and 21.5; 512: 92, 49 and 37.5.  64
// experts of about two rows each, 2048 x 2048: 41 (few) and 51 (256 columns); 16 rows: 50,
// 71 and 53; 64 rows: 91, 73 and 57.
tq_status launch_linear_f8(const F8Product &p, const DeviceInfo &dev, cudaStream_t s) {
    const int64_t experts = p.offsets ? (p.experts < p.M ? p.experts : p.M) : 1, rows = (p.M + experts - 1) / experts;
    auto cost = [&](int64_t tokens, int64_t cols, int64_t lone, int64_t other) {
        const int64_t token_tiles = (rows + tokens - 1) / tokens, tiles = experts * token_tiles * ((p.N + cols - 1) / cols);
        return (tiles + dev.sms - 1) / dev.sms * (token_tiles == 1 ? lone : other);
    };
    const int64_t few = cost(64, 128, 36 + rows / 4, 52), half = cost(128, 128, 62, 52), many = cost(128, 256, 80, 60);
    if (few <= half && few <= many) return launch_f8<false>(p, 128, dev, s);
    return launch_f8<true>(p, half < many ? 128 : 256, dev, s);
}

}  // namespace tq
