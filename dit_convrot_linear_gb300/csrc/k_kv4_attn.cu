// Attention over the 4-bit cache: o = H^T softmax(scale (H q) . k') v', with
// k' = s_k (u - 8) and v' = s_v (u - 8), u the stored nibbles.
//
// Decoding is bound by the cache's stream: dim + 8 bytes a token and key/value
// head, read once for all query heads that share it.  The kernel is one pass:
//
//   - The query rows of a sequence and key/value head (its tokens times the
//     heads that share it) are cut into row tiles of R = 8 NR, the positions a
//     row tile may see into tiles of 32.  All (sequence, head, row tile, tile)
//     quadruples, in this order, are cut into equal runs, one a group of warps
//     (a CTA's eight, or two groups of four), so ragged lengths fill the GPU
//     evenly and a single long row is split over all of it.  The lengths are read
//     on the device; each CTA finds its runs by a scan.
//   - A group's warps take turns at its tiles, each with a ring of stages of its
//     own that it fills by bulk copies (a block of 16 tokens, keys, values and
//     scales, lies in one piece) as it frees them; no warp waits for another.
//     Each keeps its own maximum, sum and output, joined in shared memory at the
//     end of a run's part in a row tile, and over CTAs through the workspace by
//     the one that comes last (in run order: the result does not depend on
//     timing).
//   - Products run on mma.sync m16n8k16: with 8 or 16 query rows against 32
//     tokens there is no 128-row tile for the tensor cores' own memory, and the
//     operands come from registers: a nibble masked out of a word is the fp16
//     subnormal u 2^-24, so a lane's 16-byte load is a whole operand row without
//     conversion; an odd nibble is used with its even neighbour left below it (u
//     + 16 u'), which the query's even element, less a sixteenth of the odd one,
//     or the output's subtraction at the end, takes out.  Tokens are the
//     rows (M) of S^T = K Q^T and the depth of O^T = V^T P^T, query rows the
//     columns, so that few rows waste little.  The bias of 8 is taken off the
//     scores by the accumulator's start value (-8 sum q) and off the output by
//     one more product with a constant operand (8 sum w).
//   - The running maximum is raised only when a score passes it by 2^8: the
//     weights then stay below 2^8 and the output is seldom rescaled.  A weight
//     times its value's scale is rounded to fp16 relative to the largest scale
//     met (2^-12 of itself, an order below the cache's own rounding); sums stay
//     in fp32.
//
// Measured (8 key/value heads of 128, 32 query heads), against the time of the
// bytes at the card's copy rate: four contexts of 131072 98 us, 84 (86 %); 64
// sequences of up to 4096 47, 25; 24 of up to 5 drafted tokens, window 4096, 51,
// 15; one of 777 tokens (14 heads of 64 on 2) 10.7, of which a launch that does
// nothing is 2 to 3.  The long ones are bound by the stream.  The others by what
// happens once a run: about 6 us until the first tile is at hand (lengths, pages
// and blocks are fetched one after the other here; only the blocks have to wait
// for the pages), 3 to 4 us where a row tile ends and the next begins, 3 to 5 us
// to join parts.  Heads 64 wide: those 64 sequences 36, 13.5, one of 777 10.8;
// 256 wide: 72, 49, and 14.3.

#include <cfloat>

#include "tq_a16.cuh"
#include "tq_kv4.cuh"

namespace tq {
namespace {

constexpr int kTile = 32;                    // tokens a tile: two blocks
constexpr int kFold = 4;                     // tiles of a warp between two subtractions of the bias
constexpr int kLeast = 16;                   // the shortest run
// Fewest tiles a part, where row tiles are cut on their own: one sequence of 40000
// on 2 heads, widths 64 / 128 / 256, 20.5 / 23.9 / 25.1 us; with 24 21.9 / 24.0 /
// 25.7, with 96 22.8 / 29.6 / 31.2 (9000 tokens: 16.6 / 19.8 / 23.2; 15.0 / 17.3 /
// 18.5; 23.9 / 30.2 / 36.8).
constexpr int kMinRun = 48;
constexpr unsigned int kStatusKvTimeout = 128u;
// A copy of the library built for its own tests lets every stage expect bytes
// that no copy brings (their waits then run out).
#ifdef TQ_TEST_UNSET_BYTES
constexpr uint32_t kUnset = TQ_TEST_UNSET_BYTES;
#else
constexpr uint32_t kUnset = 0;
#endif
constexpr float kNone = -FLT_MAX;            // running maximum before any score
constexpr float kSlack = 8.0f;               // log2 by which a score may pass it
constexpr float kLog2e = 1.4426950408889634f;

template <int D_, int NR_, int NW_, int GW_, int STAGES_, int CTAS_>
struct Cfg {
    static constexpr int D = D_, NR = NR_, NW = NW_, GW = GW_, STAGES = STAGES_, CTAS = CTAS_;
    static constexpr int G = NW / GW;                        // groups of GW warps, each with runs of its own
    static constexpr int GT = GW * 32;
    // Tiles that starting and ending a row tile stand for.  Half as many: 64
    // sequences up to 4096, widths 64 / 128 / 256, 38.5 / 49.9 / 78.0 us where these
    // take 36.1 / 47.2 / 72.5; twice as many: 35.4 / 47.2 / 76.4.
    static constexpr int OVER = 40 / G;
    static constexpr int R = 8 * NR;                         // query rows a row tile
    static constexpr int NT = NW * 32;                       // threads
    static constexpr int W = D / 32;                         // 32-bit words of a row a lane
    static constexpr bool QREG = NR * W <= 4;                // queries stay in registers
    static constexpr int BLK = kv_block_bytes(D);
    static constexpr int TILE = 2 * BLK;
    static constexpr int QROW = 2 * D + 64;                  // bytes; rows 64 bytes apart mod 128: no bank conflicts
    static constexpr int OROW = D + 4;                       // floats
    static constexpr int OBUF = R * OROW * 4;
    static constexpr int JOIN0 = (CTAS == 1 ? 67584 : 34816) / OBUF;     // output buffers: as many warps join at once
    static constexpr int JOIN = JOIN0 < 2 ? 2 : JOIN0 < NW ? JOIN0 : NW;
    // shared memory
    static constexpr int oQ = NW * STAGES * TILE;
    static constexpr int oO = oQ + (QREG ? 0 : G * R * QROW);    // (queries that go to registers lie under the output)
    static constexpr int oStat = oO + JOIN * OBUF;           // the float arrays named in the kernel
    static constexpr int oBar = oStat + (2 * R * G + 2 * NW * R) * 4;
    static constexpr int QGROUP = QREG ? GW * OBUF : R * QROW;
    static constexpr int oSeq = oBar + NW * STAGES * 8;
    static constexpr int oIter = oSeq + NT * static_cast<int>(sizeof(KvSeq));
    static constexpr int oFound = oIter + NW * 64;
    static constexpr int oPart = oFound + G * 64;
    static constexpr int oNext = oPart + G * 2 * 64;
    static constexpr int oFlag = oNext + G * 3 * 64;
    static constexpr int SMEM = oFlag + 4 * (1 + 2 * G);
    static constexpr int oScan = oO;                         // before any output
    static_assert(NW % GW == 0 && (G == 1 || JOIN == NW) && NT * 8 + NW * 8 <= JOIN * OBUF && R * QROW <= OBUF * JOIN / G && SMEM <= 228 * 1024 / CTAS - 1024, "shared memory");
};

// A row tile's weight in the cutting: its tiles, and as many as starting and
// ending a row tile takes as long as.
template <int OVER>
__device__ __forceinline__ int weight(int tiles) { return tiles ? tiles + OVER : 0; }

// Weight of all row tiles of a sequence (one head), by one thread.
template <int OVER>
__device__ __forceinline__ int64_t seq_cost(const Geo &ge, const KvSeq &q) {
    const int nrt = row_tiles(ge, q);
    int64_t sum = 0;
#pragma unroll 1
    for (int rt = 0; rt < nrt; ++rt) {
        int lo, hi, t0, c;
        range_of<kTile>(ge, q, rt, lo, hi, t0, c);
        sum += weight<OVER>(c);
    }
    return sum;
}

// The same by a warp.
template <int OVER>
__device__ __forceinline__ int64_t seq_cost_warp(const Geo &ge, const KvSeq &q) {
    const int nrt = row_tiles(ge, q), lane = threadIdx.x & 31;
    int64_t sum = 0;
    for (int rt = lane; rt < nrt; rt += 32) {
        int lo, hi, t0, c;
        range_of<kTile>(ge, q, rt, lo, hi, t0, c);
        sum += weight<OVER>(c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// The next row tile in order.  `seqs`: the sequences' descriptions in shared
// memory, where one step of the scan held them all (else nullptr).
__device__ __forceinline__ bool advance(const tq_kv4 &kv, const Geo &ge, const KvSeq *seqs, Run &u) {
    do {                                     // row tiles that see nothing are left out
        if (++u.rt >= u.nrt) {
            u.rt = 0;
            if (++u.h >= kv.heads) {
                u.h = 0;
                bool bad = false;
                do {
                    if (++u.b >= kv.nseq) return false;
                    u.q = seqs ? seqs[u.b] : kv_seq(kv, u.b, bad);
                } while (u.q.n == 0 || u.q.len == 0);
                u.nrt = row_tiles(ge, u.q);
            }
        }
        range_of<kTile>(ge, u.q, u.rt, u.lo, u.hi, u.t0, u.cost);
    } while (u.cost == 0);
    return true;
}

// A word's nibbles 0 .. 7 as fp16 pairs, in units of 2^-24 (a 16-bit pattern
// below 2^10 is that many times 2^-24): the pairs (0, 4) and (2, 6), and each
// with 16 times its neighbours (1, 5) and (3, 7) added.  Four instructions:
// taking the neighbours out would be a fifth, and is left to whoever uses them.
__device__ __forceinline__ void nibbles(uint32_t x, uint32_t &n04, uint32_t &n04_15, uint32_t &n26, uint32_t &n26_37) {
    n04_15 = x & 0x00FF00FFu;
    asm("prmt.b32 %0, %1, 0, 0x4341;" : "=r"(n26_37) : "r"(x));
    n04 = x & 0x000F000Fu;
    n26 = n26_37 & 0x000F000Fu;
}

// Transpose of an 8 x 8 matrix of 16-bit values held as mma fragments are.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int W>
__device__ __forceinline__ void lds_words(const unsigned char *p, uint32_t (&w)[W]) {
    if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    }
}

// the product as a value of its operands alone, so that the compiler may order it
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Found {                               // where a CTA's run starts
    int64_t at, head;                        // tiles of the sequence before it; tiles a head
    int b;
    KvSeq q;
};

struct Part {                                // a part of a row tile whose others are elsewhere
    Run u;
    int cf, cl;                              // CTAs that hold its parts
};
static_assert(3 * sizeof(Run) <= 192 && sizeof(Part) <= 64 && sizeof(Found) <= 64, "shared memory");

struct AttnParams {
    tq_kv4 kv;
    Kv4Attn a;
    Geo geo;
    unsigned int *count;     // [grid] arrivals, zero between calls
    float *part;             // [2 grid][R][D] partial outputs
    float *stat;             // [2 grid][R][2] their maxima (log2) and sums
    unsigned int *status;
    int min_run;             // fewest tiles a run
    int aligned;             // few row tiles: cut each on its own
    int wide;                // rows of one sequence may fill more than one row tile
};

template <class C>
__global__ void __launch_bounds__(C::NT, C::CTAS) k_kv4_attn(const __grid_constant__ AttnParams p) {
    constexpr int D = C::D, NR = C::NR, NW = C::NW, R = C::R, W = C::W, S = C::STAGES;
    constexpr int GW = C::GW, G = C::G, GT = C::GT, kOver = C::OVER;
    constexpr bool OWN = C::JOIN == NW;      // an output buffer a warp
    extern __shared__ __align__(128) unsigned char sm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t smb = smem_addr(sm);
    const int group = warp / GW, gw = warp % GW, gtid = tid % GT;
    auto group_sync = [&]() {
        if constexpr (G == 1) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(GT) : "memory");
    };
    float *rowf = reinterpret_cast<float *>(sm + C::oStat) + group * 2 * R;
    float *rowc = rowf + R;
    // each warp's maximum and sum [GW][R]
    float2 *wstat = reinterpret_cast<float2 *>(sm + C::oStat + G * 2 * R * 4) + group * GW * R;
    const uint32_t bar0 = smb + C::oBar + warp * S * 8;      // this warp's stages
    const uint32_t ring_at = smb + warp * S * C::TILE;
    int64_t *scan = reinterpret_cast<int64_t *>(sm + C::oScan);
    int64_t *wsum = scan + C::NT;
    volatile int *flag = reinterpret_cast<volatile int *>(sm + C::oFlag);   // 0: a wait ran out; two a group: last to arrive
    volatile int *came_last = flag + 1 + 2 * group;
    const tq_kv4 &kv = p.kv;
    const Geo &ge = p.geo;
    KvSeq *seqs_sh = reinterpret_cast<KvSeq *>(sm + C::oSeq);
    const KvSeq *seqs = kv.nseq <= C::NT ? seqs_sh : nullptr;
    Found *found = reinterpret_cast<Found *>(sm + C::oFound + group * 64);
    Part *parts = reinterpret_cast<Part *>(sm + C::oPart + group * 128);
    float *obuf = reinterpret_cast<float *>(sm + C::oO) + group * (OWN ? GW : 0) * (C::OBUF / 4);
    unsigned char *qsm = sm + C::oQ + group * C::QGROUP;

    if (tid == 0) {
        for (int i = 0; i < NW * S; ++i)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smb + C::oBar + 8 * i) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        flag[0] = 0;
    }

    // ---------------------------------------------------- this CTA's run
    pdl_launch_dependents();
    pdl_wait();                           // lengths, pages, queries and the workspace may come from the launch before
    bool bad = false;
    KvSeq mine = {0, 0, 0};               // sequence base + tid of the scan's step, its tiles a head, and
    int64_t head = 0, mine_at = 0, step_sum = 0;   // those of all heads before it in the step and in the step
    auto block_scan = [&](int64_t v, int64_t &before, int64_t &all) {      // exclusive prefix, and the sum
        int64_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        before = x - v;
        all = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
    };
    auto scan_step = [&](int64_t base) {
        mine = {0, 0, 0};
        if (base + tid < kv.nseq) mine = kv_seq(kv, base + tid, bad);
        seqs_sh[tid] = mine;
        if (p.wide) {                     // many row tiles: a warp a sequence
            const int here = static_cast<int>(kv.nseq - base < C::NT ? kv.nseq - base : C::NT);
            __syncthreads();
            for (int i = warp; i < here; i += NW) {
                const int64_t c = seq_cost_warp<kOver>(ge, seqs_sh[i]);
                if (lane == 0) scan[i] = c;
            }
            __syncthreads();
            head = tid < here ? scan[tid] : 0;
        } else {
            head = seq_cost<kOver>(ge, mine);
        }
        block_scan(head * kv.heads, mine_at, step_sum);
    };
    int64_t total = 0;
    for (int64_t base = 0; base < kv.nseq; base += C::NT) {
        if (base) __syncthreads();
        scan_step(base);
        total += step_sum;
    }
    if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusIndex);
    auto leave_idle = [&]() { zero_rows<D>(kv, p.a, ge); };
    const int64_t runs = static_cast<int64_t>(gridDim.x) * G;
    int64_t per = quotient(total + runs - 1, runs);
    per = per < p.min_run ? p.min_run : per;
    const int run = static_cast<int>(blockIdx.x) * G + group;
    Run u;
    int64_t uw = 0;                       // weight before the run's first row tile over the batch
    int n_all = 0;                        // the run's tiles
    int first = 0;                        // the run's first tile in its row tile
    bool aligned = false;                 // each row tile is cut on its own, into parts of about `per` tiles
    int acf = 0, acl = 0;                 // the CTAs that hold its parts then
    auto parts_of = [&](int64_t cost) { return cost < per ? cost > 0 : static_cast<int>(quotient(cost, per)); };
    if (G == 1 && p.aligned) {
        int np = 0;                       // parts of a head of this thread's sequence
        const int nrt = row_tiles(ge, mine);
        for (int rt = 0; rt < nrt; ++rt) {
            int lo, hi, t0, c;
            range_of<kTile>(ge, mine, rt, lo, hi, t0, c);
            np += parts_of(c);
        }
        int64_t np_at, np_sum;
        __syncthreads();
        block_scan(static_cast<int64_t>(np) * kv.heads, np_at, np_sum);
        aligned = np_sum <= runs;
        if (aligned) {
            if (run >= np_sum) {
                leave_idle();
                return;
            }
            const int64_t k = run - np_at;
            if (k >= 0 && k < static_cast<int64_t>(np) * kv.heads) {
                found->b = tid;
                found->q = mine;
                found->at = k;
                found->head = np;
            }
            __syncthreads();
            u.b = found->b;
            u.q = found->q;
            u.nrt = row_tiles(ge, u.q);
            u.h = static_cast<int>(found->at) / static_cast<int>(found->head);
            int k2 = static_cast<int>(found->at) % static_cast<int>(found->head), n2 = 1;
            for (u.rt = 0; u.rt < u.nrt; ++u.rt) {
                range_of<kTile>(ge, u.q, u.rt, u.lo, u.hi, u.t0, u.cost);
                n2 = parts_of(u.cost);
                if (k2 < n2) break;
                k2 -= n2;
            }
            acf = run - k2;
            acl = acf + n2 - 1;
            first = static_cast<int>(static_cast<int64_t>(u.cost) * k2 / n2);
            n_all = static_cast<int>(static_cast<int64_t>(u.cost) * (k2 + 1) / n2) - first;
        }
    }
    if (!aligned) {
        const int64_t first0 = static_cast<int64_t>(blockIdx.x) * G * per;     // of the CTA's runs
        int64_t passed = 0;
        for (int64_t base = 0; base < kv.nseq; base += C::NT) {
            if (kv.nseq > C::NT) {        // one step: its scan is still at hand
                __syncthreads();
                scan_step(base);
            }
            for (int g = 0; g < G; ++g) {
                const int64_t k = first0 + g * per - passed - mine_at;
                if (k >= 0 && k < head * kv.heads) {
                    Found *f = reinterpret_cast<Found *>(sm + C::oFound + g * 64);
                    f->b = static_cast<int>(base + tid);
                    f->q = mine;
                    f->at = k;
                    f->head = head;
                }
            }
            passed += step_sum;
            if (first0 + (G - 1) * per < passed) break;
        }
        __syncthreads();
        const int64_t c0 = run * per, c1 = c0 + per < total ? c0 + per : total;
        if (c0 >= c1) {
            leave_idle();
            return;
        }
        u.b = found->b;
        u.q = found->q;
        u.nrt = row_tiles(ge, u.q);
        u.h = static_cast<int>(quotient(found->at, found->head));
        int64_t at = found->at - u.h * found->head;
        u.rt = 0;
        if (u.nrt > 1) {                  // the row tile: by 32 at a time
            for (int base = 0; base < u.nrt; base += 32) {
                int lo, hi, t0, c = 0;
                if (base + lane < u.nrt) range_of<kTile>(ge, u.q, base + lane, lo, hi, t0, c);
                c = weight<kOver>(c);
                int64_t x = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                const unsigned in = __ballot_sync(0xffffffffu, x > at);
                if (in) {
                    const int l = __ffs(in) - 1;
                    u.rt = base + l;
                    at -= __shfl_sync(0xffffffffu, x - c, l);
                    break;
                }
                at -= __shfl_sync(0xffffffffu, x, 31);
            }
        }
        range_of<kTile>(ge, u.q, u.rt, u.lo, u.hi, u.t0, u.cost);
        // the weight of starting comes first: a run that ends within it leaves
        // the row tile to the next
        first = at > kOver ? static_cast<int>(at) - kOver : 0;
        uw = c0 - at;
        Run v = u;
        int64_t w = uw;
        for (int f = first;; f = 0) {
            const int64_t end = c1 - w - kOver;
            n_all += end > f ? (end < v.cost ? static_cast<int>(end) : v.cost) - f : 0;
            w += kOver + v.cost;
            if (w >= c1 || !advance(kv, ge, seqs, v)) break;
        }
        if (n_all == 0) {
            leave_idle();
            return;
        }
    }
    // The raw queries of the next row tile come while the tiles of this one are
    // read: a row a warp, and further ones by turns.
    constexpr int E = D / 32, RW = (R + GW - 1) / GW;
    constexpr bool AHEAD = RW <= 2;                  // (more rows would cost the registers)
    uint32_t raw[RW][E / 2];
    auto load_queries = [&](const Run &v) {
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const int row = v.rt * R + gw + k * GW;
            const bool is = gw + k * GW < R && row < v.q.n * ge.g;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                p.a.Q + static_cast<int64_t>(v.q.start + (is ? row / ge.g : 0)) * p.a.ldq +
                static_cast<int64_t>(v.h * ge.g + (is ? row % ge.g : 0)) * D + lane * E);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) raw[k][e] = is ? src[e] : 0u;
        }
    };
    if constexpr (AHEAD) load_queries(u);

    // ---------------------------------------------------- this warp's copies
    // Its tiles are gw, gw + GW, .. of the run.  Lane i holds where tile i of
    // 32 at a time lies (the number of its block in the pool plus one, two of them
    // where a page is half a tile; 0: nowhere), and the stages are filled in turn.
    uint32_t src0 = 0, src1 = 0;
    const bool halves = kv.page_size < kTile;
    {
        Run *it = reinterpret_cast<Run *>(sm + C::oIter + warp * 64);
        if (lane == 0) *it = u;
        __syncwarp();
    }
    int n_send = n_all, it_start = -first;           // the iterator's row tile begins at this tile of the run
    auto find_tiles = [&](int k0) {                  // tiles k0, k0 + GW, .. of the run
        Run *it = reinterpret_cast<Run *>(sm + C::oIter + warp * 64);
        Run v = *it;
        const int k = k0 + lane * GW, end = min(k0 + 32 * GW, n_all);
        src0 = src1 = 0;
        for (;;) {
            if (k >= it_start && k < it_start + v.cost && k < n_all) {
                const int pos = (v.t0 + k - it_start) * kTile;
                if (pos < v.hi) {
                    src0 = kv_block_number(kv, v.b, v.h, pos) + 1;
                    if (halves && pos + kKvBlock < v.hi) {
                        src1 = kv_block_number(kv, v.b, v.h, pos + kKvBlock) + 1;
                        bad |= src1 == 0;
                    }
                    bad |= src0 == 0;
                }
            }
            if (it_start + v.cost >= end) break;
            it_start += v.cost;
            if (!advance(kv, ge, seqs, v)) break;
        }
        __syncwarp();
        if (lane == 0) *it = v;
        __syncwarp();
    };
    int sent = 0;                                    // tiles copied so far
    uint32_t there = 0;                              // per stage, next one lowest: which of its blocks are there
    auto send = [&](int k, uint32_t at, uint32_t bar) {      // tile k of the run, into the stage at `at`
        uint32_t a0 = 0, a1 = 0;
        if (k < n_send) {
            if ((sent & 31) == 0) find_tiles(k);
            a0 = __shfl_sync(0xffffffffu, src0, sent & 31);
            if (halves) a1 = __shfl_sync(0xffffffffu, src1, sent & 31);
            ++sent;
            if (elect_one()) {
                const uint32_t n0 = halves ? C::BLK : C::TILE;
                const uint64_t pool = reinterpret_cast<uint64_t>(kv.pool) - C::BLK;
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                             "r"(kUnset + (a0 ? n0 : 0u) + (a1 ? C::BLK : 0u))
                             : "memory");
                if (a0) bulk_copy(at, pool + static_cast<uint64_t>(a0) * C::BLK, n0, bar);
                if (a1) bulk_copy(at + C::BLK, pool + static_cast<uint64_t>(a1) * C::BLK, C::BLK, bar);
            }
            __syncwarp();
        }
        there = (there >> 2) | (((a0 ? (halves ? 1u : 3u) : 0u) | (a1 ? 2u : 0u)) << (2 * (S - 1)));
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) send(gw + i * GW, ring_at + i * C::TILE, bar0 + 8 * i);

    // ---------------------------------------------------- parts of the run
    const int r = lane >> 2, j = lane & 3;
    int done = 0;                         // tiles of the run before this part
    int from = first;
    bool lost = false;
    uint32_t at = ring_at, bar = bar0, phase = 0;    // this warp's next stage
    int next = gw;                        // and its next tile of the part
    // Row tiles in turn.  Parts whose others are elsewhere go to the workspace;
    // at the end of the run their arrivals are counted (once, for all of them),
    // and the CTA that comes last joins them.  A row tile's parts belong to CTAs
    // cf .. cl; only the first of them can hold it as its run's last part (slot
    // 2 cf + 1), the others hold it as their run's first (slot 2 c).  Joining the
    // warps and joining the parts are one piece of code: what few CTAs run has to
    // be fetched from far away.
    int nparts = 0, joined = -1;          // parts left elsewhere; parts looked at for the last join
    int cf = 0, cl = 0;
    // the next row tile, in two places in turn (a slow warp may still read the last)
    Run *next_sh = reinterpret_cast<Run *>(sm + C::oNext + group * 192), *cur_sh = next_sh + 2;
    int turn = 0;
    for (;;) {
      const bool last = done >= n_all;    // joining parts, not warps
      bool whole = true;
      if (last) {
        if (joined < 0) {
            if (nparts == 0) break;
            group_sync();
            if (gtid == 0) {
                __threadfence();          // the CTA's stores, ordered before it by the barrier
                for (int i = 0; i < nparts; ++i) {
                    const unsigned int old = atomicAdd(p.count + parts[i].cf, 1u);
                    came_last[i] = old == static_cast<unsigned int>(parts[i].cl - parts[i].cf);
                    if (came_last[i]) p.count[parts[i].cf] = 0u;
                }
                __threadfence();
            }
            group_sync();
            joined = 0;
        }
        while (joined < nparts && !came_last[joined]) ++joined;
        if (joined == nparts) break;
        u = parts[joined].u;
        cf = parts[joined].cf;
        cl = parts[joined].cl;
        ++joined;
      } else {
        const int n = min(u.cost - from, n_all - done);
        const int rows = u.q.n * ge.g, r0 = u.rt * R;

        if constexpr (!AHEAD) load_queries(u);
        // the row tile's queries: rotated, as fp16 in the order of the words'
        // nibbles (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
        for (int k0 = 0; k0 < RW; ++k0) {
            const int i = gw + k0 * GW;
            if (R % GW && i >= R) break;
            float v[8];
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = __uint_as_float(e & 1 ? raw[k0][e / 2] & 0xFFFF0000u : raw[k0][e / 2] << 16);
            warp_fwht<E, float>(v);
            const float cn = sqrtf(1.0f / D);
            float mx = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[e] = cn * v[e];
                mx = fmaxf(mx, fabsf(v[e]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // the row's largest value in [2^13, 2^14)
            const int k = mx > 0.0f ? min(13 - (static_cast<int>(__float_as_uint(mx) >> 23) - 127), 126) : 0;
            const float up = pow2i(k);
            // an odd value's operand meets its nibble with 16 times it: over 16;
            // an even one's meets it alone once more, so that much is taken off
            float sum = 0.0f;
            unsigned char *qrow = qsm + i * C::QROW;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const int d = lane * E + e, jj = d / (D / 4), w = (d % (D / 4)) / 8, nb = d % 8;
                const __half odd = __float2half_rn(v[e + 1] * up * 0.0625f);
                const __half even = __float2half_rn(v[e] * up - __half2float(odd));
                sum += __half2float(even) + 17.0f * __half2float(odd);
                __half *dst = reinterpret_cast<__half *>(qrow + ((w * 4 + jj) * 8 + (nb & 3) * 2 + (nb >> 2)) * 2);
                dst[0] = even;
                dst[2] = odd;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) {
                rowf[i] = p.a.scale * kLog2e * (16777216.0f * pow2i(-k));
                rowc[i] = -8.0f / 16777216.0f * sum;
            }
        }
        if (done + n < n_all) {
            Run v = u;
            advance(kv, ge, seqs, v);
            if constexpr (AHEAD) load_queries(v);
            if (gtid == 0) next_sh[turn] = v;
        }
        if (gtid == 0) *cur_sh = u;
        group_sync();

        // per lane: query rows 8 nt + 2 j and 8 nt + 2 j + 1
        float f[NR][2], cst[NR][2], m[NR][2], l[NR][2];
        int all_lo = 0, all_hi = 0x7fffffff;          // positions that every row sees
        uint32_t qf[C::QREG ? NR : 1][C::QREG ? W : 1][4];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int i = nt * 8 + 2 * j + c;
                f[nt][c] = rowf[i];
                cst[nt][c] = rowc[i];
                m[nt][c] = kNone;
                l[nt][c] = 0.0f;
                if (r0 + i < rows) {
                    int lo, hi;
                    row_range(ge, u.q, (r0 + i) / ge.g, lo, hi);
                    all_lo = max(all_lo, lo);
                    all_hi = min(all_hi, hi);
                }
            }
            if constexpr (C::QREG) {
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t t4[4];
                    lds_words<4>(qsm + (nt * 8 + r) * C::QROW + (w * 4 + j) * 16, t4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) qf[nt][w][e] = t4[e];
                }
            }
        }
        if constexpr (C::QREG) group_sync();             // before any output lands there
        all_lo = __reduce_max_sync(0xffffffffu, all_lo);
        all_hi = __reduce_min_sync(0xffffffffu, all_hi);

        float o[NR][D / 16][4], oc[NR][4];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) oc[nt][e] = 0.0f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][t][e] = 0.0f;
        }
        float gv = pow2i(127);                // power of two that value scales are multiplied by

        // this warp's tiles of the part
        const int tile0 = u.t0 + from;
#pragma unroll 1
        for (; next < n; next += GW) {
            if (!mbar_try(bar, phase)) {
                if (lost || !mbar_wait_bounded(bar, phase, flag[0] ? 0 : kA16WaitLimit)) {
                    lost = true;
                    n_send = 0;           // nothing more is sent into stages that did not fill
                    flag[0] = 1;
                    if (lane == 0) atomicOr(p.status, kStatusKvTimeout);
                    continue;
                }
            }
            const int tile_at = (tile0 + next) * kTile;
            const unsigned char *base = sm + (at - smb);
            const uint32_t have = there & 3u;

            // scores: S^T, tokens r and r + 8 of each block, times the key's scale
            float s[2][NR][4], sv[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const unsigned char *blk = base + k * C::BLK;
                uint32_t x[W], y[W];
                lds_words<W>(blk + r * (D / 2) + j * (D / 8), x);
                lds_words<W>(blk + (r + 8) * (D / 2) + j * (D / 8), y);
                const float *sc = reinterpret_cast<const float *>(blk + 16 * D);
                const float sk[2] = {sc[r], sc[r + 8]};
                sv[k][0] = sc[16 + r];
                sv[k][1] = sc[24 + r];
#pragma unroll
                for (int nt = 0; nt < NR; ++nt) {
                    s[k][nt][0] = s[k][nt][2] = cst[nt][0];
                    s[k][nt][1] = s[k][nt][3] = cst[nt][1];
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                    nibbles(x[w], a0, a2, b0, b2);
                    nibbles(y[w], a1, a3, b1, b3);
#pragma unroll
                    for (int nt = 0; nt < NR; ++nt) {
                        uint32_t q4[4];
                        if constexpr (C::QREG) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) q4[e] = qf[nt][w][e];
                        } else {
                            lds_words<4>(qsm + (nt * 8 + r) * C::QROW + (w * 4 + j) * 16, q4);
                        }
                        mma(s[k][nt], a0, a1, a2, a3, q4[0], q4[1]);
                        mma(s[k][nt], b0, b1, b2, b3, q4[2], q4[3]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[k][nt][e] *= sk[e >> 1];
            }

            // a tile at the edge of what its rows see, or with a page left out
            if (!(have == 3u && tile_at >= all_lo && tile_at + kTile <= all_hi)) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = cur_sh->rt * R + nt * 8 + 2 * j + e;
                        int lo = 0, hi = 0;
                        if (row < cur_sh->q.n * ge.g) row_range(ge, cur_sh->q, row / ge.g, lo, hi);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int pos = tile_at + k * 16 + c * 8 + r;
                                if (!((have >> k) & 1u) || pos < lo || pos >= hi) s[k][nt][2 * c + e] = -INFINITY;
                            }
                    }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int pos = tile_at + k * 16 + c * 8 + r;
                        if (!((have >> k) & 1u) || pos < cur_sh->lo || pos >= cur_sh->hi) sv[k][c] = 0.0f;
                    }
            }

            // log2 of the weights, relative to the running maximum
            float ex[2][NR][4];
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ex[k][nt][e] = fmaf(s[k][nt][e], f[nt][e & 1], -m[nt][e & 1]);
                        top = fmaxf(top, ex[k][nt][e]);
                    }
            if (__any_sync(0xffffffffu, top > kSlack)) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float t = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
                        const float to = fmaxf(m[nt][c], t * f[nt][c]);
                        const float fix = ex2(m[nt][c] - to);
                        m[nt][c] = to;
                        l[nt][c] *= fix;
                        oc[nt][c] *= fix;
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            o[nt][d][c] *= fix;
                            o[nt][d][c + 2] *= fix;
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            ex[k][nt][c] = fmaf(s[k][nt][c], f[nt][c], -to);
                            ex[k][nt][c + 2] = fmaf(s[k][nt][c + 2], f[nt][c], -to);
                        }
                    }
            }
            // value scales near the top of fp16's range, the largest met below 2^7
            float big = max_nan(max_nan(sv[0][0], sv[0][1]), max_nan(sv[1][0], sv[1][1]));
            if (__any_sync(0xffffffffu, !(big * gv <= 128.0f))) {
                // a value whose scale is not finite goes into the scores of the rows
                // that see it: 0 times it would be NaN in the others' outputs
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (!(sv[k][c] <= FLT_MAX)) {
                            sv[k][c] = 0.0f;
#pragma unroll
                            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                                for (int e = 2 * c; e < 2 * c + 2; ++e)
                                    if (s[k][nt][e] != -INFINITY) ex[k][nt][e] = __uint_as_float(0x7FFFFFFFu);
                        }
                big = fmaxf(fmaxf(sv[0][0], sv[0][1]), fmaxf(sv[1][0], sv[1][1]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
                if (big * gv > 128.0f) {                 // (of the whole warp)
                    const float to = pow2i(5 - (static_cast<int>(__float_as_uint(big) >> 23) - 127));
                    const float fix = to / gv;
                    gv = to;
#pragma unroll
                    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            oc[nt][e] *= fix;
#pragma unroll
                            for (int d = 0; d < D / 16; ++d) o[nt][d][e] *= fix;
                        }
                }
            }

            // output: O^T, value words of token pairs j and j + 4
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const unsigned char *blk = base + k * C::BLK + 8 * D;
                uint32_t x[W], y[W], b0[NR], b1[NR];
                lds_words<W>(blk + j * D + r * (D / 8), x);
                lds_words<W>(blk + (j + 4) * D + r * (D / 8), y);
                const float g0 = sv[k][0] * gv, g1 = sv[k][1] * gv;
#pragma unroll
                for (int nt = 0; nt < NR; ++nt) {
                    float w4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = ex2(ex[k][nt][e]);
                        l[nt][e & 1] += w;
                        w4[e] = w * (e < 2 ? g0 : g1);
                    }
                    b0[nt] = transpose8(half2_bits(w4[0], w4[1]));
                    b1[nt] = transpose8(half2_bits(w4[2], w4[3]));
                    mma(oc[nt], 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, b0[nt], b1[nt]);
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t a0, a1, a2, a3, c0_, c1_, c2_, c3_;
                    nibbles(x[w], a0, a1, c0_, c1_);
                    nibbles(y[w], a2, a3, c2_, c3_);
#pragma unroll
                    for (int nt = 0; nt < NR; ++nt) {
                        mma(o[nt][2 * w], a0, a1, a2, a3, b0[nt], b1[nt]);
                        mma(o[nt][2 * w + 1], c0_, c1_, c2_, c3_, b0[nt], b1[nt]);
                    }
                }
            }
            // The bias comes off now and then: fp32 sums of nibbles, 8 on average,
            // outgrow those of their values by the root of the tokens, and the
            // tensor cores' truncation with them (131072 tokens: 0.0042 of the
            // output where every fourth tile leaves 0.0017, bf16's own share).
            if ((next & (kFold * GW - 1)) >= (kFold - 1) * GW) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float b = (e < 2 ? 1.0f : 17.0f) * oc[nt][e & 1];
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) o[nt][d][e] -= b;
                    }
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) oc[nt][e] = 0.0f;
            }
            // every lane's reads of the stage before the next copy into it
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            send(done + next + S * GW, at, bar);
            at += C::TILE;
            bar += 8;
            if (at == ring_at + S * C::TILE) {
                at = ring_at;
                bar = bar0;
                phase ^= 1;
            }
        }
        u = *cur_sh;

        // ------------------------------------------------ join the warps
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
                if (r == 0) wstat[gw * R + nt * 8 + 2 * j + c] = make_float2(m[nt][c], l[nt][c]);
            }
        // Each warp's output into a buffer of its own, relative to its own
        // maximum; where there are fewer buffers than warps, in rounds, relative
        // to the rows' largest.
        float up[NR][2];
        if constexpr (!OWN) group_sync();
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                up[nt][c] = 16777216.0f / gv;
                if constexpr (!OWN) {
                    float mx = kNone;
#pragma unroll
                    for (int w = 0; w < GW; ++w) mx = fmaxf(mx, wstat[w * R + nt * 8 + 2 * j + c].x);
                    up[nt][c] *= ex2(m[nt][c] - mx);
                }
            }
#pragma unroll 1
        for (int round = 0; OWN ? round < 1 : round * C::JOIN < NW; ++round) {
            if (OWN || warp / C::JOIN == round) {
                float *buf = obuf + (OWN ? gw : warp % C::JOIN) * (C::OBUF / 4);
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            float4 *dst = reinterpret_cast<float4 *>(buf + (nt * 8 + 2 * j + c) * C::OROW + r * (D / 8) + 4 * w);
                            const float b = oc[nt][c], fc = up[nt][c];
                            float4 v = make_float4((o[nt][2 * w][c] - b) * fc,
                                                   ((o[nt][2 * w][c + 2] - o[nt][2 * w][c]) * 0.0625f - b) * fc,
                                                   (o[nt][2 * w + 1][c] - b) * fc,
                                                   ((o[nt][2 * w + 1][c + 2] - o[nt][2 * w + 1][c]) * 0.0625f - b) * fc);
                            if (!OWN && round) {
                                const float4 t = *dst;
                                v = make_float4(v.x + t.x, v.y + t.y, v.z + t.z, v.w + t.w);
                            }
                            *dst = v;
                        }
            }
            group_sync();
        }

        whole = from == 0 && n == u.cost;
        if (!whole) {
            cf = aligned ? acf : static_cast<int>(quotient(uw + kOver, per));
            cl = aligned ? acl : static_cast<int>(quotient(uw + kOver + u.cost - 1, per));
            if (gtid == 0) parts[nparts] = {u, cf, cl};
            ++nparts;
        }
        done += n;
        next -= n;
        from = 0;
      }

      // L lanes join a row over its sources: the warps' buffers, or the parts (a
      // piece of a part is a trip to far memory: each lane brings as many as the
      // rings hold, empty by now, into places of its own there).
      constexpr int L0 = GT / R < D / 4 ? GT / R : D / 4;
      constexpr int L = L0 >= 32 ? 32 : L0 >= 16 ? 16 : 8, V = D / L;   // lanes a row, values a lane
      constexpr int DEPTH = GW * S * C::TILE / (GT * 4 * V);
      static_assert(DEPTH >= 1 && L >= GW, "one step joins the warps");
      const uint32_t gring = smb + group * GW * S * C::TILE;
      const bool keep = last || whole;
      const bool scaled = last || OWN;                   // else the buffers share the largest maximum
      const int np = last ? cl - cf + 1 : GW, no = scaled ? np : C::JOIN;
      const float2 *st = reinterpret_cast<const float2 *>(p.stat) + static_cast<int64_t>(2) * cf * R;
      constexpr int sstep = 2 * R, sfirst = R;
      const int64_t slot = 2 * static_cast<int64_t>(run) + (run == cf ? 1 : 0);
      const int rows = u.q.n * ge.g, r0 = u.rt * R, sub = lane % L;
#pragma unroll 1
      for (int base = gw * (32 / L); base < R && r0 + base < rows; base += GT / L) {
        const int i = base + lane / L;
        const bool is = r0 + i < rows;                   // (a last row without a partner: its lanes go along)
        auto bring = [&](int k0, int n) {
            const float *src = p.part + static_cast<int64_t>(2) * cf * (R * D) + i * D + sub * V;
#pragma unroll 1
            for (int k = 0; k < n; ++k) {
                const int kk = k0 + k;
                const float *from_ = src + static_cast<int64_t>(kk ? 2 * kk : 1) * (R * D);
                const uint32_t to = gring + (k * GT + gtid) * (4 * V);
#pragma unroll
                for (int e = 0; e < V; e += 4)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 4 * e), "l"(from_ + e) : "memory");
            }
        };
        if (last) bring(0, min(no, DEPTH));
        // (another join on this SM may have left a line with this one's statistics
        // in L1 before they were written: past it)
        auto stat = [&](int k) { return last ? __ldcg(st + k * sstep + (k ? 0 : sfirst) + i) : wstat[k * R + i]; };
        float mx = kNone;
#pragma unroll 1
        for (int k = sub; k < np; k += L) mx = fmaxf(mx, stat(k).x);
#pragma unroll
        for (int x = 1; x < L; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        float sum = 0.0f, v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.0f;
#pragma unroll 1
        for (int k0 = 0, in = 0; k0 < np; k0 += L) {     // `in`: sources brought before this step's
            float fac = 0.0f;
            if (k0 + sub < np) {
                const float2 t2 = stat(k0 + sub);
                fac = ex2(t2.x - mx);
                sum = fmaf(fac, t2.y, sum);
            }
            if (!scaled) fac = 1.0f;
            const int n = min(L, no - k0);
#pragma unroll 4
            for (int k = 0; k < n; ++k) {
                const float *src;
                if (last) {
                    const int at_ = (k0 + k) - in;
                    if (at_ == DEPTH) {
                        in += DEPTH;
                        bring(in, min(no - in, DEPTH));
                    }
                    if (at_ == 0 || at_ == DEPTH) asm volatile("cp.async.wait_all;" ::: "memory");
                    src = reinterpret_cast<const float *>(sm + (gring - smb) + ((k0 + k - in) * GT + gtid) * (4 * V));
                } else {
                    src = obuf + k * (C::OBUF / 4) + i * C::OROW + sub * V;
                }
                const float f = __shfl_sync(0xffffffffu, fac, k, L);
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = fmaf(f, src[e], v[e]);
            }
        }
#pragma unroll
        for (int x = 1; x < L; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (!keep) {                                     // to the workspace
            float *dst = p.part + (slot * R + i) * D + sub * V;
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<float4 *>(dst + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            if (sub == 0) reinterpret_cast<float2 *>(p.stat)[slot * R + i] = make_float2(mx, sum);
            continue;
        }
        const bool none = sum <= 0.0f;                   // (a NaN sum is not: it goes on to the output)
        const float inv = none ? 0.0f : sqrtf(1.0f / D) / sum;
#pragma unroll
        for (int h = 1; h < V; h <<= 1)                  // turned back
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (!(e & h)) {
                    const float a = v[e], b = v[e + h];
                    v[e] = a + b;
                    v[e + h] = a - b;
                }
#pragma unroll
        for (int x = 1; x < L; x <<= 1)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float b = __shfl_xor_sync(0xffffffffu, v[e], x);
                v[e] = sub & x ? b - v[e] : v[e] + b;
            }
        uint32_t w[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) w[e] = none ? 0u : bf16_bits2(v[2 * e] * inv, v[2 * e + 1] * inv);
        if (flag[0] || !is) continue;                    // the sums are not whole
        const int64_t tok = u.q.start + (r0 + i) / ge.g;
        const int hq = u.h * ge.g + (r0 + i) % ge.g;
        uint16_t *dst = p.a.O + tok * p.a.ldo + static_cast<int64_t>(hq) * D + sub * V;
        if constexpr (V == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        else
#pragma unroll
            for (int e = 0; e < V / 2; e += 4)
                *reinterpret_cast<uint4 *>(dst + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
        if (p.a.lse && sub == 0)
            p.a.lse[tok * p.a.heads_q + hq] = none ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
      }
      group_sync();
      if (!last && done < n_all) {
        uw += u.cost + kOver;
        u = next_sh[turn];
        turn ^= 1;
      }
    }
    zero_rows<D>(kv, p.a, ge);
    if (bad) atomicOr(p.status, kStatusIndex);
    if (lost && lane == 0) {
        // after a wait that ran out nobody has seen the copies land: wait for
        // the last use of each of this warp's stages
        const long long t0 = clock64();
        for (int i = 0; i < S && i < sent; ++i) {
            const long long left = kA16DrainLimit - (clock64() - t0);
            mbar_wait_bounded(bar0 + 8 * i, ((sent - 1 - i) / S) & 1, left > 0 ? left : 0);
        }
    }
}

constexpr int kMaxSlots = 8;                             // parts an SM (two a run), over the variants
constexpr int kMaxPart = 8 * 8 * 128;                    // slots an SM times R times D, over the variants
constexpr int kMaxStat = 8 * 16;                         // slots an SM times R
size_t count_bytes(const DeviceInfo &dev) { return (static_cast<size_t>(dev.sms) * kMaxSlots / 2 * 4 + 255) / 256 * 256; }

template <class C>
tq_status launch(AttnParams &p, const DeviceInfo &dev, cudaStream_t s) {
    static_assert(2 * C::CTAS * C::G <= kMaxSlots && 2 * C::CTAS * C::G * C::R * C::D <= kMaxPart && 2 * C::CTAS * C::G * C::R <= kMaxStat, "workspace");
    const int grid = dev.sms * C::CTAS;
    unsigned char *ws = static_cast<unsigned char *>(p.a.ws);
    p.count = reinterpret_cast<unsigned int *>(ws);
    p.stat = reinterpret_cast<float *>(ws + count_bytes(dev));
    p.part = p.stat + static_cast<size_t>(dev.sms) * kMaxStat * 2;
    p.geo.rows = C::R;
    p.wide = p.a.max_q * p.geo.g > 4 * C::R;
    // Row tiles, if max_q is right: where there are several CTAs for each, each
    // is cut into parts of its own (at least kMinRun tiles, so a short context
    // is not cut at all: joining parts costs 4 us, a tile 0.1); else all tiles
    // into equal runs, of at least one a warp.
    const int64_t tiles = p.kv.nseq * p.kv.heads * ((p.a.max_q * p.geo.g + C::R - 1) / C::R);
    p.aligned = C::G == 1 && p.kv.nseq <= C::NT && tiles * 4 <= grid;
    p.min_run = p.aligned ? kMinRun : kLeast;
    const cudaError_t fe = cudaFuncSetAttribute(k_kv4_attn<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_kv4_attn<C>, p);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e);
}

}  // namespace

size_t kv4_workspace_bytes(const DeviceInfo &dev) {
    const size_t runs = count_bytes(dev) + static_cast<size_t>(dev.sms) * (2 * kMaxStat + kMaxPart) * 4;
    const size_t tc = kv4_tc_workspace_bytes(dev);
    return (runs + 255) / 256 * 256 + tc;
}

tq_status launch_kv4_attention(const tq_kv4 &kv, const Kv4Attn &a, const DeviceInfo &dev, cudaStream_t s) {
    AttnParams p = {};
    p.kv = kv;
    p.a = a;
    p.geo.g = a.heads_q / kv.heads;
    p.geo.causal = a.causal;
    p.geo.window = a.window;
    p.status = status_word();
    if (!p.status) return TQ_ERR_DEVICE;
    const int64_t rows = a.max_q * p.geo.g;
    if (kv4_tc_takes(kv, a, rows)) {
        const size_t runs = count_bytes(dev) + static_cast<size_t>(dev.sms) * (2 * kMaxStat + kMaxPart) * 4;
        return launch_kv4_attention_tc(kv, a, static_cast<unsigned char *>(a.ws) + (runs + 255) / 256 * 256, dev, s);
    }
    // Up to 8 rows at a time, or 16 (rows beyond them are further row tiles).  32
    // at once took 107 us where two times 16 took 63 (24 sequences of up to 5
    // drafted tokens, window 4096): its accumulators leave a warp no room to
    // overlap.  Where there are more than a quarter as many row tiles as SMs, two
    // groups of four warps a CTA with runs of their own, so that one starts or
    // ends a row tile while the other streams: those drafts 50 us against 56, 64
    // sequences of up to 4096 47 against 52, 256 of up to 700 59 against 78.
    // With fewer, all eight warps on one part: 4 contexts of 131072 97 us against
    // 104, one of 777 10.5 against 12.5.  (Groups of two: 48, 57, 60, 113, 19.)
    // Heads 64 wide, groups of four against eight warps: 64 sequences up to 4096
    // 36 and 41, 256 up to 700 47 and 64, the drafts 38 and 41; 4 of 65536 48 and
    // 40, one of 777 12.7 and 10.9.  256 wide: 72 and 84, 100 and 134; one of 777
    // 16.8 and 14.3, but 4 of 65536 97 and 100.
    const bool wide = rows > 8;
    const int64_t tiles = kv.nseq * kv.heads * ((rows + (wide ? 15 : 7)) / (wide ? 16 : 8));
    const bool many = 4 * tiles > dev.sms;
    if (kv.dim == 64) {
        if (wide) return many ? launch<Cfg<64, 2, 8, 4, 3, 2>>(p, dev, s) : launch<Cfg<64, 2, 8, 8, 3, 2>>(p, dev, s);
        return many ? launch<Cfg<64, 1, 8, 4, 4, 2>>(p, dev, s) : launch<Cfg<64, 1, 8, 8, 4, 2>>(p, dev, s);
    }
    if (kv.dim == 128) {
        if (wide) return many ? launch<Cfg<128, 2, 8, 4, 3, 1>>(p, dev, s) : launch<Cfg<128, 2, 8, 8, 4, 1>>(p, dev, s);
        return many ? launch<Cfg<128, 1, 8, 4, 2, 2>>(p, dev, s) : launch<Cfg<128, 1, 8, 8, 2, 2>>(p, dev, s);
    }
    if (wide) return launch<Cfg<256, 2, 8, 8, 2, 1>>(p, dev, s);     // (no room for a buffer a warp)
    return many ? launch<Cfg<256, 1, 8, 4, 2, 1>>(p, dev, s) : launch<Cfg<256, 1, 8, 8, 2, 1>>(p, dev, s);
}

}  // namespace tq
