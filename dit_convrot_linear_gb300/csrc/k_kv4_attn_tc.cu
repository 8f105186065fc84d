// Attention over the 4-bit cache for many query rows a key/value head (a
// prompt's chunk, drafted tokens), on tcgen05: o = H^T softmax(scale (H q) . k') v'.
//
// With tens to thousands of rows the products bound the kernel, and mma.sync
// reaches about a quarter of the tensor cores' rate here (9.1 cycles an
// m16n8k16 measured, 520 TFLOP/s).  A CTA takes row tiles of one or two times
// 128 query rows (a sequence's tokens times the heads that share a key/value
// head) against tiles of 128 positions:
//
//   - a loader warp copies blocks of 16 tokens into a ring;
//   - eight warps widen them to fp16 operands in shared memory, a block of a tile
//     each, without a word between them: a nibble put under 1024's exponent is
//     1024 + u (or 1024 + 16 u), from which u - 8 comes exactly, times s, the
//     token's scale over a power of two of the block's largest.  (A nibble taken
//     as the subnormal u 2^-24 saves that step, but its product with s is among
//     fp16's subnormals from a scale 2^-4 of the block's largest on: 0.8 % off at
//     2^-8.  As it is, the product keeps its 11 bits down to 2^-25.)
//     Keys are the K-major rows of S = Q K^T; values, whose words hold two tokens,
//     are the K-major rows of O = P V as they come;
//   - one thread issues the products: S into TMEM (128 columns a row tile), P
//     (fp16, over S's columns) times V into O, also in TMEM.  With two row tiles
//     one's softmax runs during the other's products; with one, S has two places;
//   - two threads a row do the softmax, 64 positions each: the scores come from
//     TMEM, twice (the maximum, which the two exchange, then the weights, which go
//     back over them).  The running maximum is raised only when passed by 2^8; O
//     is then rescaled in place, which the tensor cores' order of work makes safe.
//     (One pass that takes the maximum for granted until a score passes it by 2^15
//     took 351 us where two take 322: a vote every 16 columns.)
//
// The row tiles stand in a line, each as long as its tiles and a few for its start
// and end, and every CTA takes an equal piece of it; a second kernel joins the
// parts of those that were cut, a warp a row, in order (the result does not depend
// on timing).  Sums and statistics are fp32; q, k', p and v' are rounded to fp16
// relative to their row's, block's or maximum's scale.
//
// Measured (8 key/value heads of 128, 32 query heads): 1024 rows over 16384
// tokens 307 us, 139 for their operations at a large library product's rate (mma.sync
// took 1056); the last 4096 rows of as many 1004 us, 503; four prompts of 4096 830,
// 288.  Heads of 64: 268 us, 70.  A pair of row tiles takes about 4900 cycles a tile
// of positions where its products alone would take 2050: a row tile's softmax (2900)
// and its products (1700, slowed by the widening warps' stores: both operands of S
// come from shared memory, all of its bandwidth) follow one another, and TMEM has no
// room for a second set of scores beside two outputs.

#include <cfloat>

#include "tq_a16.cuh"
#include "tq_kv4.cuh"

namespace tq {
namespace {

constexpr int kTileT = 128;                  // positions a tile
constexpr int kHalf = 64;                    // positions copied and widened at a time
constexpr int kBlocks = kHalf / kKvBlock;    // blocks of them
constexpr int kRing = 3;                     // halves in the ring
// Barriers of their arrival: two a stage, in turn, so that each serves the warps
// of one half alone (a wait tells only two neighbouring phases apart, and the
// warps that take every second use of a stage would miss one between).
constexpr int kFull = 2 * kRing;
constexpr unsigned int kStatusKvTcTimeout = 256u;
constexpr float kNoneT = -FLT_MAX;
constexpr float kSlackT = 8.0f;
constexpr float kLog2eT = 1.4426950408889634f;
constexpr int kMaxSeqsT = 256;               // sequences the cutting holds in shared memory
constexpr int kNoE = -1024;                  // exponent of a half whose values are all zero
constexpr int kCols = 512;                   // TMEM columns
constexpr int kMaxSmsT = 160;                // more SMs than this stay unused
// Tiles that a part's start and end stand for: 64 rows over 16384, widths 64 / 128,
// 40.7 / 51.4 us, eight prompts of 2000 435 / 554; with 2 39.4 / 50.6 and 450 / 577,
// with 8 49.1 / 60.0 and 447 / 551.
constexpr int kStart = 4;
constexpr int kMinPart = 4;                  // fewest tiles a part

// A build for the library's own tests expects bytes that no copy brings.
#ifdef TQ_TEST_UNSET_BYTES
constexpr uint32_t kUnset = TQ_TEST_UNSET_BYTES;
#else
constexpr uint32_t kUnset = 0;
#endif

template <int D_, int NQ_>
struct TCfg {
    static constexpr int D = D_, NQ = NQ_;
    static constexpr int RU = 128 * NQ;                      // query rows a row tile
    static constexpr int WSM = 8 * NQ;                       // softmax warps: two for the same 32 rows, half the columns each
    static constexpr int W_DQ = WSM, W_LD = WSM + 8, W_MMA = WSM + 9;
    static constexpr int NT = (WSM + 10) * 32;
    static constexpr int BLK = kv_block_bytes(D);
    static constexpr int RAW = kBlocks * BLK;
    static constexpr int KT = kTileT * D * 2;                // bytes of a key tile, of a value tile, of a query tile
    static constexpr int oK = 0, oV = 2 * KT, oQ = 4 * KT, oRaw = oQ + NQ * KT;
    static constexpr int oBar = oRaw + kRing * RAW;
    static constexpr int USED = oBar + 32 * 8;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;       // one CTA an SM: it takes all of TMEM
};

struct Item {                                // a CTA's part of a row tile
    int n, at, lo, hi;                       // tiles, its first position; positions of the row tile
    int slot;                                // where its sums go (-1: it is the whole row tile)
    int b, h, rt;
    bool last;                               // it ends its row tile
    int64_t next;                            // where the CTA goes on
    KvSeq q;
};

// What the join knows of a CTA: whether its first part goes on with the row tile
// of the CTA before (1) and ends it (2); whether its last one begins a row tile
// that the next CTA goes on with (4), and which.
struct Cut {
    int flags, start, rows, h, rt, pad[3];
};

struct TcParams {
    tq_kv4 kv;
    Kv4Attn a;
    Geo geo;
    unsigned int *status;
    int ctas;                                // of the attention kernel
    Cut *table;                              // [grid]
    float2 *stat;                            // [2 grid][RU]
    float *part;                             // [2 grid][RU][D]
};

__device__ __forceinline__ uint32_t sa(const void *p) { return smem_addr(p); }

// A bounded wait by a whole warp, with one answer for all its lanes.  On expiry
// the CTA's flag is raised, and every wait ends at once from then on; the roles
// run through their loops without work, so that no barrier is left waiting.  A
// role that has given up waits and arrives no more: a barrier that stands still
// has always completed one of the two parities, and an arrival too many faults.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *status) {
    bool ok = mbar_try(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const long long t0 = clock64();
        while (!ok) {
            ok = mbar_try(bar, parity);
            if (ok || *abort) break;
            if (clock64() - t0 > kA16WaitLimit) {
                *abort = 1;
                atomicOr(status, kStatusKvTcTimeout);
            }
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// K-major operand of 8x8 core matrices, 64 columns a panel (rows * 128 bytes)
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46);
}

#define TQ_R32(v)                                                                                                 \
    "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), \
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]),           \
        "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]),           \
        "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])

__device__ __forceinline__ void t_ld32(uint32_t at, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(at));
}

__device__ __forceinline__ void t_st32(uint32_t at, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        TQ_R32(v));
}

__device__ __forceinline__ void t_ld16(uint32_t at, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
}

__device__ __forceinline__ void t_ld8(uint32_t at, uint32_t *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
}

__device__ __forceinline__ void t_st8(uint32_t at, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]));
}

// The loaded registers are operands of the wait, so that no use of them moves
// before it.
__device__ __forceinline__ void t_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void t_wait_ld(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void t_wait_ld(uint32_t (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void t_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// a b + c of fp16 pairs (exact but for one rounding), and a b
__device__ __forceinline__ uint32_t hfma2_(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t hmul2_(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ unsigned long long pair2(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void split2(unsigned long long r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// u - 8, u = 0 .. 15 in bits 0 .. 3 (FAR: bits 4 .. 7) of both halves of x, the
// others zero: 1024 + u less 1032, or (1024 + 16 u) / 16 less 72
constexpr uint32_t k1024 = 0x64006400u, kOne = 0x3C003C00u, kMinus1032 = 0xE408E408u;
constexpr uint32_t kSixteenth = 0x2C002C00u, kMinus72 = 0xD480D480u;
template <bool FAR>
__device__ __forceinline__ uint32_t code_of(uint32_t x) {
    return FAR ? hfma2_(x | k1024, kSixteenth, kMinus72) : hfma2_(x | k1024, kOne, kMinus1032);
}

constexpr float kWide = 2048.0f;             // widened keys and values are this many times what they stand for

template <class C>
__global__ void __launch_bounds__(C::NT, 1) k_kv4_attn_tc(const __grid_constant__ TcParams p) {
    constexpr int D = C::D, NQ = C::NQ, RU = C::RU, PAN = kTileT * 128;      // PAN: bytes of a 64-column panel of 128 rows
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ uint32_t tmem_sh;
    __shared__ volatile int abort_sh;
    __shared__ int64_t run_sh[2], before_sh[kMaxSeqsT + 1];      // before: of all heads of the sequences before
    __shared__ KvSeq seq_sh[kMaxSeqsT];
    struct __align__(16) Info {              // of a block: 2^e / kWide of the keys, exponent of the values (read as a
        float kx;                            // pair: first, at 16 bytes); whether it is there
        int ev;
        int there, pad;
    };
    __shared__ uint32_t raw_there[kRing];
    __shared__ float rowf_sh[RU];                            // a row's factor
    // What a row's two threads exchange: their maxima, and their sums.  A row's own
    // place serves both: its two warps alone keep step.  The maxima stay in fp32:
    // a bound above them by log2 units (16 bits of a score of thousands are off by
    // tens) would leave the weights below fp16's range.  With two row tiles one
    // place a half serves every tile: tile k + 1's scores come only after both
    // warps have handed over tile k's weights, and so have read its maxima; with
    // one they come ahead, so there are two places in turn.
    constexpr int PLACES = NQ == 2 ? 1 : 2;
    __shared__ union { float max[PLACES][2]; float sum[2]; } pair_sh[RU];
    __shared__ Info kv_info[4][8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const tq_kv4 &kv = p.kv;
    const Geo &ge = p.geo;
    const uint32_t smb = sa(sm);
    const uint32_t bar = smb + C::oBar;
    const uint32_t raw_full = bar, raw_empty = bar + 48, k_full = bar + 72, k_empty = bar + 88, v_full = bar + 104,
                   v_empty = bar + 120, s_full = bar + 136, p_full = bar + 152, q_full = bar + 168, pv_done = bar + 184,
                   all_done = bar + 200;

    if (tid == 0) {
        auto init = [&](uint32_t b, int n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(n) : "memory");
        };
        for (int i = 0; i < kFull; ++i) init(raw_full + 8 * i, 1);
        for (int i = 0; i < kRing; ++i) init(raw_empty + 8 * i, 4);
        for (int i = 0; i < 2; ++i) {
            init(k_full + 8 * i, 8);
            init(k_empty + 8 * i, 1);
            init(v_full + 8 * i, 8);
            init(v_empty + 8 * i, 1);
            init(s_full + 8 * i, 1);
            init(p_full + 8 * i, 8);
            init(q_full + 8 * i, 8);
            init(pv_done + 8 * i, 1);
        }
        init(all_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_sh = 0;
    }
    if (warp == C::W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&tmem_sh)), "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_launch_dependents();
    pdl_wait();

    // ---------------------------------------------------- cutting
    // The row tiles stand in a line, each as long as its tiles and kStart; a CTA
    // takes an equal piece of it.  First the lengths (a warp a sequence).
    const int nseq = static_cast<int>(kv.nseq);
    bool bad = false;
    for (int i = tid; i < nseq; i += C::NT) seq_sh[i] = kv_seq(kv, i, bad);
    if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusIndex);
    __syncthreads();
    for (int i = warp; i < nseq; i += C::NT / 32) {
        const KvSeq q = seq_sh[i];
        const int nrt = row_tiles(ge, q);
        int64_t sum = 0;
        for (int rt = lane; rt < nrt; rt += 32) {
            int lo, hi, t0, c;
            range_of<kTileT>(ge, q, rt, lo, hi, t0, c);
            if (c > 0) sum += c + kStart;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) before_sh[i + 1] = sum * kv.heads;
    }
    if (tid == 0) before_sh[0] = 0;
    __syncthreads();
    if (warp == 0) {                             // running sums
        int64_t run = 0;
        for (int base = 0; base < nseq; base += 32) {
            int64_t x = base + lane < nseq ? before_sh[base + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (base + lane < nseq) before_sh[base + lane + 1] = run + x;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_sh;

    // The row tile at `x` of the line, by a whole warp; where it begins, and its
    // tiles and the first of them.
    auto find = [&](int64_t x, Item &it, int64_t &begin, int &t0, int &tiles) {
        int lo = 0, hi = nseq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before_sh[mid] <= x) lo = mid;
            else hi = mid;
        }
        it.b = lo;
        it.q = seq_sh[lo];
        const int64_t each = quotient(before_sh[lo + 1] - before_sh[lo], kv.heads);
        int64_t k = x - before_sh[lo];
        it.h = static_cast<int>(quotient(k, each));
        k -= it.h * each;
        const int nrt = row_tiles(ge, it.q);
        it.rt = 0;
        for (int base = 0; base < nrt; base += 32) {
            int l1 = 0, h1 = 0, c = 0;
            if (base + lane < nrt) range_of<kTileT>(ge, it.q, base + lane, l1, h1, t0, c);
            const int n = c > 0 ? c + kStart : 0;
            int s = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            const unsigned in = __ballot_sync(0xffffffffu, s > k);
            if (in) {
                const int l = __ffs(in) - 1;
                it.rt = base + l;
                k -= __shfl_sync(0xffffffffu, s - n, l);
                break;
            }
            k -= __shfl_sync(0xffffffffu, s, 31);
        }
        begin = x - k;
        range_of<kTileT>(ge, it.q, it.rt, it.lo, it.hi, t0, tiles);
    };
    // This CTA's piece: from the warps 0 and 1, its two ends.  An end with fewer
    // than kMinPart tiles of its row tile on one side moves to that side.
    if (warp < 2) {
        const int64_t total = before_sh[nseq];
        const int64_t runs = min(static_cast<int64_t>(gridDim.x), max(quotient(total, kStart + kMinPart), int64_t{1}));
        int64_t x = total;
        if (blockIdx.x + warp < runs) {
            x = quotient(total * (blockIdx.x + warp), runs);
            if (x < total) {
                Item it;
                int64_t begin;
                int t0, tiles;
                find(x, it, begin, t0, tiles);
                const int64_t in = x - begin - kStart;
                if (in < kMinPart) x = begin;
                else if (tiles - in < kMinPart) x = begin + kStart + tiles;
            }
        }
        if (lane == 0) run_sh[warp] = x;
    }
    __syncthreads();
    const int64_t run0 = run_sh[0], run1 = run_sh[1];

    // The part of a row tile that begins at `x`.
    auto item = [&](int64_t x) {
        Item it;
        int64_t begin;
        int t0, tiles;
        find(x, it, begin, t0, tiles);
        const int from = x == begin ? 0 : static_cast<int>(x - begin - kStart);
        const int64_t end = begin + kStart + tiles;
        const int to = run1 >= end ? tiles : static_cast<int>(run1 - begin - kStart);
        it.n = to - from;
        it.at = (t0 + from) * kTileT;
        it.slot = from > 0 ? 2 * static_cast<int>(blockIdx.x) : to < tiles ? 2 * static_cast<int>(blockIdx.x) + 1 : -1;
        it.last = to == tiles;
        it.next = min(run1, end);
        return it;
    };

    if (warp == C::W_LD) {
        // ------------------------------------------------ loader
        int k = 0, sent = 0;                     // halves
        bool ok = true;
        for (int64_t x = run0; x < run1;) {
            const Item it = item(x);
            x = it.next;
            for (int t = 0; t < 2 * it.n; ++t, ++k) {
                const int s = k % kRing;
                const int at = it.at + t * kHalf;
                // a copy a page's piece of the half: lane 0 .. 3 a block each, the
                // first of a page's for all of them
                const int each = min(kBlocks, kv.page_size / kKvBlock);
                uint32_t num = 0;
                const int pos = at + (lane / each * each) * kKvBlock;
                if (lane < kBlocks && pos < it.hi) {
                    num = kv_block_number(kv, it.b, it.h, pos) + 1;
                    if (num == 0) bad = true;
                }
                const uint32_t there = __ballot_sync(0xffffffffu, num != 0) & ((1u << kBlocks) - 1);
                ok = ok && tc_wait(raw_empty + 8 * s, ((k / kRing) & 1) ^ 1, &abort_sh, p.status);
                if (!ok) continue;
                if (lane == 0) {
                    raw_there[s] = there;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(raw_full + 8 * (k % kFull)),
                                 "r"(static_cast<uint32_t>(__popc(there)) * C::BLK + kUnset)
                                 : "memory");
                    ++sent;
                }
                __syncwarp();
                if (num && lane % each == 0)
                    bulk_copy(smb + C::oRaw + s * C::RAW + lane * C::BLK,
                              reinterpret_cast<uint64_t>(kv.pool) + static_cast<uint64_t>(num - 1) * C::BLK,
                              each * C::BLK, raw_full + 8 * (k % kFull));
                __syncwarp();
            }
        }
        if (bad) atomicOr(p.status, kStatusIndex);
        if (lane == 0)                           // never leave with copies landing
            for (int i = sent > kRing ? sent - kRing : 0; i < sent; ++i)
                mbar_wait_bounded(raw_full + 8 * (i % kFull), (i / kFull) & 1, kA16DrainLimit);
        __syncwarp();
    } else if (warp >= C::W_DQ && warp < C::W_DQ + 8) {
        // ------------------------------------------------ widening
        const int dw = warp - C::W_DQ;                           // block dw of each tile
        const int row = lane % kKvBlock, part = lane / kKvBlock; // two lanes a token
        int k = 0;
        bool ok = true;
        for (int64_t x = run0; x < run1;) {
            const Item it = item(x);
            x = it.next;
            for (int i = 0; i < it.n; ++i, ++k) {
                const int kh = 2 * k + dw / kBlocks, rs = kh % kRing, s = k & 1;
                const uint32_t par = ((k >> 1) & 1) ^ 1;
                ok = ok && tc_wait(raw_full + 8 * (kh % kFull), (kh / kFull) & 1, &abort_sh, p.status);
                if (!ok) continue;
                const unsigned char *blk = sm + C::oRaw + rs * C::RAW + (dw % kBlocks) * C::BLK;
                const bool there = (raw_there[rs] >> (dw % kBlocks)) & 1u;
                // the token's scales, and the block's largest
                const int pos = it.at + i * kTileT + kKvBlock * dw + row;
                const bool is = there && pos >= it.lo && pos < it.hi;
                const float *sc = reinterpret_cast<const float *>(blk + 16 * D);
                // (a key or value whose scale is not finite is NaN in its scores, which
                // reach the rows that see it: 0 times the value would be NaN in others)
                const bool fine = !is || (sc[row] <= FLT_MAX && sc[16 + row] <= FLT_MAX);
                const float sk = is && fine ? sc[row] : 0.0f, sv = is && fine ? sc[16 + row] : 0.0f;
                const uint32_t mk = __reduce_max_sync(0xffffffffu, __float_as_uint(sk)) >> 23;   // scales are not negative
                const uint32_t mv = __reduce_max_sync(0xffffffffu, __float_as_uint(sv)) >> 23;
                const int ek = mk ? static_cast<int>(mk) - 127 : 0, ev = mv ? static_cast<int>(mv) - 127 : kNoE;
                // scales over the power of two of the largest: 7 times one stays below 2^15
                const __half hk = fine ? __float2half_rn(sk * pow2i(-ek) * kWide) : __ushort_as_half(0x7FFF);
                const __half hv = __float2half_rn(sv * pow2i(-ev) * kWide);
                // keys: 8 nibbles to 16 bytes in the order (0, 4), (1, 5), (2, 6), (3, 7)
                ok = tc_wait(k_empty + 8 * s, par, &abort_sh, p.status);
                if (ok) {
                    if (lane == 0) kv_info[k & 3][dw] = {pow2i(ek) * (1.0f / kWide), ev, there, 0};
                    const __half2 h2 = __half2half2(hk);
                    const uint32_t s1 = *reinterpret_cast<const uint32_t *>(&h2);
                    const int r = kKvBlock * dw + row;
                    unsigned char *dst = sm + C::oK + s * C::KT + ((r >> 3) << 10) + (r & 7) * 16;
                    const uint4 *src = reinterpret_cast<const uint4 *>(blk + row * (D / 2));
#pragma unroll
                    for (int c0 = 0; c0 < D / 64; ++c0) {
                        // (from a chunk by the row, so that eight rows read different banks)
                        const int c = ((row >> (D == 128 ? 1 : 2)) + part * (D / 64) + c0) & (D / 32 - 1);
                        const uint4 x4 = src[c];
                        const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t y = x[e] >> 8;
                            const uint4 o = make_uint4(
                                hmul2_(code_of<false>(x[e] & 0x000F000Fu), s1), hmul2_(code_of<true>(x[e] & 0x00F000F0u), s1),
                                hmul2_(code_of<false>(y & 0x000F000Fu), s1), hmul2_(code_of<true>(y & 0x00F000F0u), s1));
                            const int ch = c * 4 + e;            // 8 columns
                            *reinterpret_cast<uint4 *>(dst + (ch >> 3) * PAN + (ch & 7) * 128) = o;
                        }
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) arrive(k_full + 8 * s);
                }
                // values: a lane a column, eight tokens at a time: its nibble of
                // four words, each two tokens
                ok = ok && tc_wait(v_empty + 8 * s, par, &abort_sh, p.status);
                if (ok) {
                    const int sh = (lane & 3) * 4;
                    const uint32_t own = __half_as_ushort(hv);
                    const uint32_t two = own | (__shfl_down_sync(0xffffffffu, own, 1) << 16);    // of even lanes
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        uint32_t s1[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) s1[q] = __shfl_sync(0xffffffffu, two, 8 * o + 2 * q);
                        const unsigned char *vb = blk + 8 * D + o * 4 * D;
                        unsigned char *dst = sm + C::oV + s * C::KT + (dw >> 2) * (D * 128) + (2 * (dw & 3) + o) * 128;
#pragma unroll
                        for (int d0 = 0; d0 < D; d0 += 32) {
                            const int d = d0 + lane;
                            uint32_t r[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t w = *reinterpret_cast<const uint32_t *>(vb + q * D + (d >> 2) * 4);
                                r[q] = hmul2_(code_of<false>((w >> sh) & 0x000F000Fu), s1[q]);
                            }
                            *reinterpret_cast<uint4 *>(dst + ((d >> 3) << 10) + (d & 7) * 16) = make_uint4(r[0], r[1], r[2], r[3]);
                        }
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        arrive(v_full + 8 * s);
                        arrive(raw_empty + 8 * rs);
                    }
                }
            }
        }
    } else if (warp == C::W_MMA) {
        // ------------------------------------------------ products
        constexpr uint32_t kIdS = (1u << 4) | (static_cast<uint32_t>(kTileT >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
        constexpr uint32_t kIdO = (1u << 4) | (static_cast<uint32_t>(D >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
        int k = 0, ni = 0;
        bool issued = false;
        auto score = [&](int q, int slot, int s) {       // S[slot] = Q[q] K[s]^T
            fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * PAN + (kk & 3) * 256;
                    const uint64_t ad = operand(smb + C::oQ + q * C::KT + off), bd = operand(smb + C::oK + s * C::KT + off);
                    asm volatile(
                        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem + slot * 128),
                        "l"(ad), "l"(bd), "r"(kIdS), "r"(kk > 0 ? 1u : 0u));
                }
                commit(s_full + 8 * slot);
            }
            __syncwarp();
        };
        auto weigh = [&](int q, int slot, int s, bool first) {   // O[q] += P[slot] V[s]
            fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTileT / 16; ++kk) {
                    const uint64_t bd = operand(smb + C::oV + s * C::KT + (kk >> 2) * (D * 128) + (kk & 3) * 256);
                    asm volatile(
                        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem + 256 + q * 128),
                        "r"(tmem + slot * 128 + (kk >> 2) * 64 + (kk & 3) * 8), "l"(bd), "r"(kIdO),
                        "r"(first && kk == 0 ? 0u : 1u));
                }
                commit(pv_done + 8 * q);
            }
            __syncwarp();
        };
        auto release = [&](uint32_t b) {
            if (elect_one()) commit(b);
            __syncwarp();
        };
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && tc_wait(b, parity, &abort_sh, p.status); };
        for (int64_t x = run0; x < run1; ++ni) {
            const Item it = item(x);
            x = it.next;
            for (int q = 0; q < NQ; ++q) wait(q_full + 8 * q, ni & 1);
            wait(k_full + 8 * (k & 1), (k >> 1) & 1);
            if (ok) {
                issued = true;
                if constexpr (NQ == 2) {
                    score(0, 0, k & 1);
                    score(1, 1, k & 1);
                } else {
                    score(0, k & 1, k & 1);
                }
                release(k_empty + 8 * (k & 1));
            }
            for (int i = 0; i < it.n; ++i, ++k) {
                const int s = k & 1, s2 = s ^ 1;
                const bool more = i + 1 < it.n;
                if constexpr (NQ == 1) {
                    if (more) {                          // the next scores during this softmax
                        wait(k_full + 8 * s2, ((k + 1) >> 1) & 1);
                        if (ok) {
                            score(0, s2, s2);
                            release(k_empty + 8 * s2);
                        }
                    }
                    wait(v_full + 8 * s, (k >> 1) & 1);
                    wait(p_full + 8 * s, (k >> 1) & 1);
                    if (ok) {
                        weigh(0, s, s, i == 0);
                        release(v_empty + 8 * s);
                    }
                } else {
                    wait(v_full + 8 * s, (k >> 1) & 1);
                    wait(p_full, k & 1);
                    if (ok) weigh(0, 0, s, i == 0);
                    if (more) {
                        wait(k_full + 8 * s2, ((k + 1) >> 1) & 1);
                        if (ok) score(0, 0, s2);
                    }
                    wait(p_full + 8, k & 1);
                    if (ok) {
                        weigh(1, 1, s, i == 0);
                        release(v_empty + 8 * s);
                        if (more) {
                            score(1, 1, s2);
                            release(k_empty + 8 * s2);
                        }
                    }
                }
            }
        }
        if (issued) {                                    // every product ends before TMEM is freed
            release(all_done);
            if (lane == 0) mbar_wait_bounded(all_done, 0, kA16DrainLimit);
            __syncwarp();
        }
    } else if (warp < C::WSM) {
        // ------------------------------------------------ softmax: two threads a row
        const int q = warp >> 3, wq = warp & 3, hc = (warp >> 2) & 1, row = q * 128 + wq * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t o_at = tmem + lanes + 256 + q * 128;
        Cut cut = {};                                    // (warp 0 keeps it)
        // the two warps of the same rows (both come by whatever has run out)
        auto pair_bar = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + q * 4 + wq) : "memory"); };
        int k = 0;
        bool ok = true;
        // Product k - 1 with the values has ended.  With two row tiles, tile k's
        // scores tell; with one they come ahead of it, and it is waited for before
        // tile k's weights are handed over: a wait tells only two neighbouring
        // phases apart, so none may be left out, nor come when the next has ended.
        auto product_before = [&]() { ok = ok && (k == 0 || tc_wait(pv_done + 8 * q, (k - 1) & 1, &abort_sh, p.status)); };
        for (int64_t x = run0; x < run1;) {
            const Item it = item(x);
            x = it.next;
            const int rows = it.q.n * ge.g, r0 = it.rt * RU;
            if (it.slot == 2 * static_cast<int>(blockIdx.x)) cut.flags = it.last ? 3 : 1;
            else if (it.slot >= 0) cut = {cut.flags | 4, it.q.start, rows, it.h, it.rt, {0, 0, 0}};
            // queries: eight lanes a row, rotated, as fp16 with the row's largest
            // value in [2^13, 2^14), eight columns in the keys' order
            const int mine = min(32, max(0, rows - (r0 + q * 128 + wq * 32)));     // rows of this warp
#pragma unroll 1
            for (int g4 = 16 * hc; g4 < 16 * hc + 16; g4 += 4) {
                constexpr int N = D / 8;
                const int rr = g4 + lane / 8, l8 = lane & 7;
                const int i = r0 + q * 128 + wq * 32 + rr;
                float v[N];
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = 0.0f;
                if (g4 < mine) {                         // (a warp's empty rows are zeros)
                    if (rr < mine) {
                        const uint16_t *src = p.a.Q + static_cast<int64_t>(it.q.start + i / ge.g) * p.a.ldq +
                                              static_cast<int64_t>(it.h * ge.g + i % ge.g) * D + l8 * N;
#pragma unroll
                        for (int e = 0; e < N; e += 8) {
                            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src + e));
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                v[e + 2 * c] = __uint_as_float(w[c] << 16);
                                v[e + 2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
                            }
                        }
                    }
                    turn_row<N>(v);
                }
                float mx = 0.0f;
#pragma unroll
                for (int e = 0; e < N; ++e) mx = fmaxf(mx, fabsf(v[e]));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const int ke = mx > 0.0f ? min(13 - (static_cast<int>(__float_as_uint(mx) >> 23) - 127), 126) : 0;
                const float up = pow2i(ke);
                const int r = wq * 32 + rr;
                if (l8 == 0) rowf_sh[q * 128 + r] = fmaxf(p.a.scale * kLog2eT * pow2i(-ke), FLT_MIN);
                unsigned char *dst = sm + C::oQ + q * C::KT + ((r >> 3) << 10) + (r & 7) * 16;
#pragma unroll
                for (int e = 0; e < N; e += 8) {
                    const uint4 o = make_uint4(half2_bits(v[e] * up, v[e + 4] * up), half2_bits(v[e + 1] * up, v[e + 5] * up),
                                               half2_bits(v[e + 2] * up, v[e + 6] * up), half2_bits(v[e + 3] * up, v[e + 7] * up));
                    const int ch = (l8 * N + e) / 8;
                    *reinterpret_cast<uint4 *>(dst + (ch >> 3) * PAN + (ch & 7) * 128) = o;
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) arrive(q_full + 8 * q);
            pair_bar();                                  // the rows' factors, of both warps
            const float f = rowf_sh[row];
            int rlo = 0, rhi = 0;
            const bool is = r0 + row < rows;
            if (is) row_range(ge, it.q, (r0 + row) / ge.g, rlo, rhi);
            const int wlo = __reduce_max_sync(0xffffffffu, is ? rlo : 0), whi = __reduce_min_sync(0xffffffffu, is ? rhi : 0x7fffffff);
            float m = kNoneT, l = 0.0f;
            int E = 0;
            for (int i = 0; i < it.n; ++i, ++k) {
                const int slot = NQ == 2 ? q : k & 1;
                const uint32_t par = NQ == 2 ? k & 1 : (k >> 1) & 1;
                ok = ok && tc_wait(s_full + 8 * slot, par, &abort_sh, p.status);
                fence_after();
                if (mine > 0) {
                    const uint32_t s_at = tmem + lanes + slot * 128 + 64 * hc;       // this warp's columns
                    const int at = it.at + i * kTileT + 64 * hc;
                    const Info *in = kv_info[k & 3];
                    const uint32_t there = __ballot_sync(0xffffffffu, lane < 8 && in[lane & 7].there) >> (4 * hc);
                    const int evm = __reduce_max_sync(0xffffffffu, in[lane & 7].ev);
                    in += 4 * hc;
                    float t = -INFINITY;
                    if (ok) {
                        if (!((there & 15u) == 15u && at >= wlo && at + 64 <= whi)) {    // what the row does not see
#pragma unroll 1
                            for (int c = 0; c < 2; ++c) {
                                uint32_t v[32];
                                t_ld32(s_at + 32 * c, v);
                                t_wait_ld(v);
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const int pos = at + 32 * c + e;
                                    if (pos < rlo || pos >= rhi || !((there >> (2 * c + e / kKvBlock)) & 1u))
                                        v[e] = 0xFF800000u;
                                }
                                t_st32(s_at + 32 * c, v);
                            }
                            t_wait_st();
                        }
                        // the largest score, in units of log2
                        uint32_t v[2][16];
                        t_ld16(s_at, v[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            t_wait_ld(v[c & 1]);
                            if (c < 3) t_ld16(s_at + 16 * (c + 1), v[(c + 1) & 1]);
                            float t0 = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) t0 = max3(t0, __uint_as_float(v[c & 1][e]), __uint_as_float(v[c & 1][e + 1]));
                            t = fmaxf(t, t0 * in[c].kx);
                        }
                        t *= f;
                    }
                    pair_sh[row].max[k % PLACES][hc] = t;
                    pair_bar();
                    t = fmaxf(t, pair_sh[row].max[k % PLACES][hc ^ 1]);
                    // E: an exponent that no value's scale passes (4 times the
                    // first ones', so that it is seldom raised)
                    const bool newE = i == 0 || evm > E;
                    if (ok && __any_sync(0xffffffffu, newE || t - m > kSlackT)) {
                        const int E0 = E;
                        if (newE) E = evm == kNoE ? -126 : evm + 2;
                        const float to = fmaxf(m, t), fix = ex2(m - to);
                        m = to;
                        l *= fix;
                        if (i > 0) {
                            if constexpr (NQ == 1) product_before();
                            fence_after();
                            const float of = fix * pow2i(E0 - E);
                            if (ok)
#pragma unroll 1
                                for (int c = hc; c < D / 32; c += 2) {       // every other piece of O
                                    uint32_t v[32];
                                    t_ld32(o_at + 32 * c, v);
                                    t_wait_ld(v);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * of);
                                    t_st32(o_at + 32 * c, v);
                                }
                            t_wait_st();
                        }
                    }
                    // the weights, over the scores already read
                    if (ok) {
                        uint32_t v[2][16];
                        t_ld16(s_at, v[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            t_wait_ld(v[c & 1]);
                            if (c < 3) t_ld16(s_at + 16 * (c + 1), v[(c + 1) & 1]);
                            const float2 ke = *reinterpret_cast<const float2 *>(&in[c].kx);
                            const int ei = __float_as_int(ke.y), ed = ei == kNoE ? 0 : max(ei - E, -100);    // <= 0
                            const float F = fmaxf(f * ke.x, FLT_MIN), dm = static_cast<float>(ed) - m;
                            const unsigned long long f2 = pair2(F, F), m2 = pair2(dm, dm);
                            unsigned long long s2 = pair2(0.0f, 0.0f);
                            uint32_t pk[8];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                unsigned long long x2;
                                asm("fma.rn.f32x2 %0, %1, %2, %3;"
                                    : "=l"(x2)
                                    : "l"(pair2(__uint_as_float(v[c & 1][e]), __uint_as_float(v[c & 1][e + 1]))), "l"(f2), "l"(m2));
                                float x0, x1;
                                split2(x2, x0, x1);
                                const float w0 = ex2(x0), w1 = ex2(x1);
                                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s2) : "l"(pair2(w0, w1)));
                                pk[e / 2] = half2_bits(w0, w1);
                            }
                            float s0, s1;
                            split2(s2, s0, s1);
                            l = fmaf(s0 + s1, pow2i(-ed), l);
                            t_st8(s_at + 8 * c, pk);
                        }
                    }
                    t_wait_st();
                }
                if constexpr (NQ == 1) product_before();
                fence_before();
                __syncwarp();
                if (lane == 0 && ok) arrive(p_full + 8 * slot);
            }
            // the output: O is whole once the last product has ended
            product_before();
            fence_after();
            if (mine > 0) {
                pair_bar();                              // the last maxima have been read
                pair_sh[row].sum[hc] = l;
                pair_bar();
                l += pair_sh[row].sum[hc ^ 1];
                if (it.slot >= 0) {
                    const float up = pow2i(E) * (1.0f / kWide);
                    if (is && hc == 0) p.stat[static_cast<int64_t>(it.slot) * RU + row] = make_float2(m, l);
                    if (ok)
#pragma unroll 1
                        for (int c = hc; c < D / 32; c += 2) {
                            uint32_t v[32];
                            t_ld32(o_at + 32 * c, v);
                            t_wait_ld(v);
                            float *dst = p.part + (static_cast<int64_t>(it.slot) * RU + row) * D + 32 * c;
                            if (is)
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    *reinterpret_cast<float4 *>(dst + e) =
                                        make_float4(__uint_as_float(v[e]) * up, __uint_as_float(v[e + 1]) * up,
                                                    __uint_as_float(v[e + 2]) * up, __uint_as_float(v[e + 3]) * up);
                        }
                } else {
                    // turn back: the butterfly over the 32-column pieces, eight
                    // columns of each at a time, then inside each piece
                    constexpr int P = D / 32;
                    if (ok)
#pragma unroll 1
                        for (int c = 16 * hc; c < 16 * hc + 16; c += 8) {
                            uint32_t v[P][8];
#pragma unroll
                            for (int b = 0; b < P; ++b) t_ld8(o_at + 32 * b + c, v[b]);
#pragma unroll
                            for (int b = 0; b < P; ++b) t_wait_ld(v[b]);
#pragma unroll
                            for (int h = 1; h < P; h <<= 1)
#pragma unroll
                                for (int b = 0; b < P; ++b)
                                    if (!(b & h))
#pragma unroll
                                        for (int e = 0; e < 8; ++e) {
                                            const float x = __uint_as_float(v[b][e]), y = __uint_as_float(v[b + h][e]);
                                            v[b][e] = __float_as_uint(x + y);
                                            v[b + h][e] = __float_as_uint(x - y);
                                        }
#pragma unroll
                            for (int b = 0; b < P; ++b) t_st8(o_at + 32 * b + c, v[b]);
                            t_wait_st();
                        }
                    fence_before();
                    pair_bar();
                    fence_after();
                    const bool none = l <= 0.0f;             // (a NaN sum is not: it goes on to the output)
                    const float inv = none ? 0.0f : sqrtf(1.0f / D) / l * pow2i(E) * (1.0f / kWide);
                    const int64_t tok = it.q.start + (is ? (r0 + row) / ge.g : 0);
                    const int hq = it.h * ge.g + (r0 + row) % ge.g;
                    uint16_t *dst = p.a.O + tok * p.a.ldo + static_cast<int64_t>(hq) * D;
                    if (ok)
#pragma unroll 1
                        for (int c = hc; c < P; c += 2) {
                            uint32_t v[32];
                            t_ld32(o_at + 32 * c, v);
                            t_wait_ld(v);
#pragma unroll
                            for (int h = 1; h < 32; h <<= 1)
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(e & h)) {
                                        const float x = __uint_as_float(v[e]), y = __uint_as_float(v[e + h]);
                                        v[e] = __float_as_uint(x + y);
                                        v[e + h] = __float_as_uint(x - y);
                                    }
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = none ? 0u : bf16_bits2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
                            if (is)
#pragma unroll
                                for (int e = 0; e < 16; e += 4)
                                    *reinterpret_cast<uint4 *>(dst + 32 * c + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                        }
                    if (is && hc == 0 && ok && p.a.lse)
                        p.a.lse[tok * p.a.heads_q + hq] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                }
            }
            fence_before();
            pair_bar();                                  // both have read O, and pair_sh
        }
        if (warp == 0 && lane == 0) p.table[blockIdx.x] = cut;
    }
    zero_rows<D>(kv, p.a, ge);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == C::W_MMA)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
}

// Joins the parts of row tiles that were cut: a warp a row.
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv4_join(const __grid_constant__ TcParams p) {
    constexpr int E = D / 32;
    __shared__ int list[kMaxSmsT], flags[kMaxSmsT], n_sh;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < p.ctas; i += kThreads) flags[i] = p.table[i].flags;
    __syncthreads();
    if (warp == 0) {                             // the row tiles that were cut, in order
        int n = 0;
        for (int base = 0; base < p.ctas; base += 32) {
            const bool begins = base + lane < p.ctas && (flags[base + lane] & 4);
            const unsigned in = __ballot_sync(0xffffffffu, begins);
            if (begins) list[n + __popc(in & ((1u << lane) - 1))] = base + lane;
            n += __popc(in);
        }
        if (lane == 0) n_sh = n;
    }
    __syncthreads();
    const int ru = p.geo.rows, g = p.geo.g, work = n_sh * ru;
    for (int w = blockIdx.x * (kThreads / 32) + warp; w < work; w += gridDim.x * (kThreads / 32)) {
        const int cta = list[w / ru], i = w % ru;
        const Cut sp = p.table[cta];
        if (sp.rt * ru + i >= sp.rows) continue;
        int np = 1;                              // parts: the last of this CTA, the first of the next ones
        while (cta + np < p.ctas && flags[cta + np++] == 1) {}
        auto slot = [&](int k) { return static_cast<int64_t>(k ? 2 * (cta + k) : 2 * cta + 1); };
        const float2 *st = p.stat + i;
        const float *src = p.part + static_cast<int64_t>(i) * D + lane * E;
        const int64_t so = ru, po = static_cast<int64_t>(ru) * D;
        float mx = kNoneT;
        for (int k = lane; k < np; k += 32) mx = fmaxf(mx, st[slot(k) * so].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float sum = 0.0f, v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll 4
        for (int k = 0; k < np; ++k) {
            const float2 t = st[slot(k) * so];
            const float f = ex2(t.x - mx);
            sum = fmaf(f, t.y, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = fmaf(f, src[slot(k) * po + e], v[e]);
        }
        warp_fwht<E, float>(v);
        const bool none = sum <= 0.0f;
        const float inv = none ? 0.0f : sqrtf(1.0f / D) / sum;
        const int row = sp.rt * ru + i;
        const int64_t tok = sp.start + row / g;
        const int hq = sp.h * g + row % g;
        uint16_t *dst = p.a.O + tok * p.a.ldo + static_cast<int64_t>(hq) * D + lane * E;
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) o[e] = none ? 0u : bf16_bits2(v[2 * e] * inv, v[2 * e + 1] * inv);
        if constexpr (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
        else *reinterpret_cast<uint32_t *>(dst) = o[0];
        if (p.a.lse && lane == 0)
            p.a.lse[tok * p.a.heads_q + hq] = none ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
    }
}

constexpr int kMaxD = 128;

template <class C>
tq_status launch(TcParams &p, void *ws, const DeviceInfo &dev, cudaStream_t s) {
    const int grid = dev.sms < kMaxSmsT ? dev.sms : kMaxSmsT;
    unsigned char *at = static_cast<unsigned char *>(ws);
    p.table = reinterpret_cast<Cut *>(at);
    p.stat = reinterpret_cast<float2 *>(at + kMaxSmsT * sizeof(Cut));
    p.part = reinterpret_cast<float *>(at + kMaxSmsT * (sizeof(Cut) + 2 * C::RU * sizeof(float2)));
    p.geo.rows = C::RU;
    p.ctas = grid;
    const cudaError_t fe = cudaFuncSetAttribute(k_kv4_attn_tc<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (fe != cudaSuccess) return cuda_fail(fe);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::NT);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k_kv4_attn_tc<C>, p);
    if (e != cudaSuccess) return cuda_fail(e);
    cfg.gridDim = dim3(grid * 8);                // (1024 rows over 16384: half as many took 5 us longer)
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, k_kv4_join<C::D>, p);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace

size_t kv4_tc_workspace_bytes(const DeviceInfo &dev) {
    (void)dev;
    return kMaxSmsT * (sizeof(Cut) + 2 * 256 * (sizeof(float2) + kMaxD * sizeof(float)));
}

// From 33 query rows a key/value head on: 64 tokens of four query heads a key/value
// head over 16384 41 us against 58 on mma.sync (heads 64 wide), 1024 268 against
// 629, or 307 against 1056 (128 wide).  Where many sequences have few rows each this
// is not so: 24 sequences of up to 9 drafted tokens (36 query rows), window 4096, 106
// us against 66 (128 wide), 91 against 46 (64), of up to 16 tokens 91 against 59.  Heads 256 wide (a row tile's output and two
// places of scores would fill TMEM) and more than 256 sequences (the cutting's arrays
// in shared memory) have no form here and run on mma.sync: 1024 rows over 16384, 256
// wide, 1760 us, 279 for their operations; 300 sequences of 16 tokens up to 700 484,
// where 256 take 316 here.
bool kv4_tc_takes(const tq_kv4 &kv, const Kv4Attn &a, int64_t rows) {
    (void)a;
    return kv.dim <= kMaxD && kv.nseq <= kMaxSeqsT && rows > 32;
}

tq_status launch_kv4_attention_tc(const tq_kv4 &kv, const Kv4Attn &a, void *ws, const DeviceInfo &dev, cudaStream_t s) {
    TcParams p = {};
    p.kv = kv;
    p.a = a;
    p.geo.g = a.heads_q / kv.heads;
    p.geo.causal = a.causal;
    p.geo.window = a.window;
    p.status = status_word();
    if (!p.status) return TQ_ERR_DEVICE;
    const bool two = a.max_q * p.geo.g > 128;
    if (kv.dim == 64) return two ? launch<TCfg<64, 2>>(p, ws, dev, s) : launch<TCfg<64, 1>>(p, ws, dev, s);
    return two ? launch<TCfg<128, 2>>(p, ws, dev, s) : launch<TCfg<128, 1>>(p, ws, dev, s);
}

}  // namespace tq
