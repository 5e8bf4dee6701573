// Dense MLA over a block-table paged latent cache for a batch whose requests
// share a prefix ("spark_model/layers/glm5next_dsa/mod.rs": the serve path's
// block-table paged MLA decode, walking 0..seq_len instead of a selected-index
// row).
//
//   z_t = sm_scale <q, kv_t>,   out = sum_t e^z_t v_t / sum_t e^z_t,   lse = log sum_t e^z_t
// over the tokens t that a (query, head) row sees; v_t are the first 512 channels of the
// row kv_t. With m the running maximum (lazily kept: within 2^8 of the true one), l the
// running sum and O the running sum of e^(z_t - m) v_t, a further token multiplies l and O
// by e^(m - m') where m grows to m'; two parts (m, l, O) merge the same way, so a sequence
// may be cut anywhere.
//
// Row tile: 64 (query, head) rows, of one query's heads or of up to four queries of fewer
// heads. Rows that share tokens thus share the copies of them: the prefix is read once for
// a tile's queries (and by the 148 CTAs together from L2), and draft tokens of one request
// share their history. Unit: 32 tokens, on the fifth-generation tensor cores
//   S[64 x 32]     = Q K^T       M = 64, N = 32;  Q's first 384 channels in tensor memory
//   O^T[512 x 64] += V^T P^T     4 blocks of M = 128, N = 64, from the same copy of the rows:
// a row is K (K-major) and V (MN-major) of one swizzled tile. Persistent: one CTA an SM,
// which works out on the device which units of which row tiles are its own (pm_plan).
//
// What bounds it: the tensor cores read their operands from shared memory at 128 bytes a
// cycle, which for tiles of 64 rows takes 1075 cycles a unit with rope (S 24 x 16.4 + 12 x
// 24.5, PV 8 x 48.5), and the copies write it too. A unit takes about 1300 cycles, in E4M3
// 1800 (the codes pass through shared memory once more and are widened there): a cache of
// half the bytes takes 5 to 40 % more time than a bf16 one of the same lengths. 64 requests
// of 128 heads behind 16384 tokens take 367 to 384 us, 0.8 PFLOP/s at the 1.6 GHz that the
// power cap leaves; 64 ragged E4M3 requests up to 32768 tokens 259 us. A request of one row
// tile over 131072 tokens is bound by HBM instead (4 of them 108 to 123 us, 4.4 to 5 TB/s). Short calls
// are bound by latencies: 2.5 us from the lengths to the plan, 1 to the first page-table
// lookups, 2 to 4 for the first units (every SM's ring fills at once: 27 to 29 MB in bf16), 1.5 to the
// first weights; behind the last product 3 us for a part's 128 KB and 6 for the second
// launch that merges the parts. One row of 512 tokens 11.9 us, 16 requests behind 6144 37.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "latent_append.cuh"
#include "sparse_mla.cuh"
#include "tc_ptx.cuh"
#include "tma.cuh"

namespace dsa {

constexpr int kMaxTokens = INT32_MAX - 64;            // a unit's last token stays an int

struct PrefixGeom {
    const int32_t *prefix_table;      // pages of the shared prefix
    const int32_t *prefix_len;        // [1] tokens of it
    const int32_t *block_table;       // [B, max_blocks] pages of each request
    const int32_t *seq_len, *q_req, *q_pos;
    int prefix_blocks, max_blocks, page, Q, B;
    int kv_rows;
    int page_shift;                   // log2(page), -1 where page is no power of two

    // Tokens of the prefix that its pages can hold.
    DSA_DEVINL int shared_len() const {
        if (prefix_blocks == 0) return 0;
        const long long cap = (long long)prefix_blocks * page;
        return (int)max(0ll, min((long long)prefix_len[0], min(cap, (long long)kMaxTokens)));
    }
    // Tokens 0 .. n-1 that a query at position pos of a sequence of len tokens sees; no
    // more than its pages can hold.
    DSA_DEVINL int visible(int pos, int len, int P) const {
        const long long n = min((long long)pos + 1, (long long)len);
        const long long cap = max((long long)P, min((long long)max_blocks * page, (long long)kMaxTokens));
        return (int)max(0ll, min(n, cap));
    }
    // Cache row of token t of the request whose pages are `pages`, -1 where there is none.
    DSA_DEVINL int row(const int32_t *pages, int t, int P) const {
        const int bi = page_shift >= 0 ? t >> page_shift : t / page;
        if (t >= P && bi >= max_blocks) return -1;
        const int blk = __ldg((t < P ? prefix_table : pages) + bi);
        const long long r = (long long)blk * page + (t - bi * page);
        return blk >= 0 && r < (long long)kv_rows ? (int)r : -1;
    }
};

// ---------------------------------------------------------------------------------------
// Row tiles and their units of work
// ---------------------------------------------------------------------------------------
constexpr int kPmTile = 32;                           // tokens of a unit: one S product
constexpr int kPmRows = 64;                           // (query, head) rows of a row tile
constexpr int kPmGrid = 148;                          // persistent CTAs, one per SM
constexpr int kPmMinUnits = 2;                        // units a CTA takes at least
constexpr int kPmPartUnits = 8;                       // units that a further part of a CTA costs
// Threads: 4 softmax warps, 8 loaders, the S and PV issuers, and a second S issuer for bf16,
// two fetchers for E4M3.
constexpr int pm_threads(bool fp8) { return fp8 ? 512 : 480; }
constexpr int kPmIssuer = 12;
constexpr int kPmQueries = 4;                         // queries a row tile holds at most

// How (query, head) rows are cut into row tiles: qpt queries of Hm < 64 heads
// each, or groups of 64 heads of one query.
struct RowTiles {
    int Hm, qpt, groups, count, total_rows;
    __host__ __device__ RowTiles(int Q, int hm)
        : Hm(hm), qpt(hm < kPmRows ? kPmRows / hm : 1), groups((hm + kPmRows - 1) / kPmRows),
          count(qpt > 1 ? (Q + qpt - 1) / qpt : Q * groups), total_rows(Q * hm) {}
    DSA_DEVINL int first_query(int t) const { return qpt > 1 ? t * qpt : t / groups; }
    DSA_DEVINL int first_row(int t) const {
        return qpt > 1 ? t * qpt * Hm : t / groups * Hm + t % groups * kPmRows;
    }
    DSA_DEVINL int rows(int t) const {
        return qpt > 1 ? min(qpt * Hm, total_rows - t * qpt * Hm)
                       : min(kPmRows, Hm - t % groups * kPmRows);
    }
};

// The tokens a row tile walks, in segments: the shared prefix (all rows); then, for
// queries of one request that follow one another, the whole units that all of them
// see (their rows), and each query's rest (its rows). With one query there is one
// segment, its whole sequence. A query that sees only a part of the prefix makes the
// tile walk without that segment. Units lie at multiples of 32 tokens, so a unit's
// rows are whole pages or parts of them.
struct TileWalk {
    int nq, npre, units, active;
    bool shared;
    int vis[kPmQueries], req[kPmQueries];
    int common[kPmQueries];           // tokens below which query k walks with its run (a multiple of 32)
    int runs;                         // 4 bits a query: queries of the run that it begins, 0 where it begins none

    DSA_DEVINL int run(int k) const { return (runs >> (4 * k)) & 15; }
    // Segment 2k: the common units of the run that begins with query k; 2k + 1: the rest of query k.
    DSA_DEVINL int segment_units(int j, int P) const {
        const int k = j >> 1;
        const unsigned base = shared ? (unsigned)P : 0u, from = max(base, (unsigned)common[k]) / kPmTile;
        if (!(j & 1)) return run(k) > 1 && (unsigned)common[k] > base ? (int)(from - base / kPmTile) : 0;
        return (unsigned)vis[k] > max(base, (unsigned)common[k])
                   ? (int)(((unsigned)vis[k] + kPmTile - 1) / kPmTile - from) : 0;
    }
    DSA_DEVINL void load(const PrefixGeom &g, const RowTiles &rt, int t, int P) {
        const int q0 = rt.first_query(t);
        nq = min(rt.qpt, g.Q - q0);
        shared = rt.qpt > 1 && P > 0;
        active = 0;
        int pos[kPmQueries], len[kPmQueries];
#pragma unroll
        for (int k = 0; k < kPmQueries; ++k) {
            req[k] = k < nq ? g.q_req[q0 + k] : -1;
            pos[k] = k < nq ? g.q_pos[q0 + k] : 0;
        }
#pragma unroll
        for (int k = 0; k < kPmQueries; ++k) {
            const bool in = req[k] >= 0 && req[k] < g.B;
            len[k] = in ? g.seq_len[req[k]] : 0;
        }
#pragma unroll
        for (int k = 0; k < kPmQueries; ++k) {
            vis[k] = g.visible(pos[k], len[k], P);
            active |= (vis[k] > 0 ? 1 : 0) << k;
            shared = shared && (vis[k] == 0 || vis[k] >= P);
        }
        shared = shared && active != 0;
        npre = shared ? (int)(((unsigned)P + kPmTile - 1) / kPmTile) : 0;
        // runs of queries of one request that all see something
        runs = 0;
        int start = 0, len_run = 0, least = 0;
#pragma unroll
        for (int k = 0; k < kPmQueries; ++k) {
            const bool joins = k > 0 && len_run > 0 && vis[k] > 0 && req[k] == req[k - 1];
            least = joins ? min(least, vis[k]) : vis[k];
            len_run = joins ? len_run + 1 : vis[k] > 0 ? 1 : 0;
            start = joins ? start : k;
            runs = (runs & ~(15 << (4 * start))) | (len_run << (4 * start));
#pragma unroll
            for (int i = 0; i < kPmQueries; ++i)
                if (i <= k && i >= start) common[i] = len_run > 1 ? least / kPmTile * kPmTile : 0;
        }
        units = npre;
#pragma unroll
        for (int j = 0; j < 2 * kPmQueries; ++j) units += segment_units(j, P);
        units = max(units, 1);                        // a tile without tokens still writes its rows
    }
};

// What a ring slot holds, written by its loader for the issuers and the softmax.
struct UnitInfo {
    // first row | rows << 8 that see these tokens | kUnit* << 16 | queries that see any token << 24
    uint32_t word;
    uint32_t valid;                                   // tokens of the unit that exist
    int part;                                         // partial slot, -1: the tile is whole
    int pad;

    DSA_DEVINL uint32_t row0() const { return word & 255u; }
    DSA_DEVINL uint32_t rows() const { return (word >> 8) & 255u; }
    DSA_DEVINL bool is(uint32_t flag) const { return (word & flag) != 0; }
};
// First and last unit of the part; rows not yet summed; rows copied without TMA; the
// part's number modulo 4.
enum : uint32_t { kUnitFirst = 1u << 16, kUnitLast = 2u << 16, kUnitFresh = 4u << 16, kUnitCopied = 8u << 16,
                  kUnitPart = 16u << 16 };

struct MergeEntry { int tile, first_cta, parts, pad; };

constexpr int kPmSBufs = 2;                           // S buffers in tensor memory
constexpr uint32_t kPmSCol = 256;                     // behind O^T
// Tensor memory's other columns hold the queries' first 384 channels: S reads
// them there instead of 2 KB of shared memory a K-step, and shared memory's
// 128 bytes a cycle are what bounds S, PV and the copies together.
constexpr int kPmQSteps = 24;                         // K-steps of 16 channels, 8 columns each
constexpr uint32_t kPmQCol = kPmSCol + kPmSBufs * kPmTile;
constexpr int kPmQChannels = kPmQSteps * 16;
constexpr uint32_t kPmAtom = kPmTile * 128;           // 64 channels of a slot's rows
constexpr uint32_t kPmPBytes = kPmRows * 128;         // two P buffers, the halves of 128-byte rows
static_assert(kPmQCol + kPmQSteps * 8 <= 512, "tensor memory columns");
constexpr int kPmMaxSlots = 6;
constexpr int kPmMaxStages = 4;
constexpr uint32_t kPmSleepNs = 100000;               // hint of a wait that may sleep

constexpr int kPlanWarps = (kPmGrid + 31) / 32;       // whose threads have row tiles that CTAs are given to

struct PmCtl {
    uint64_t kv_full[kPmMaxSlots], kv_empty[kPmMaxSlots];
    uint64_t s_full[kPmSBufs], s_empty[kPmSBufs];
    uint64_t p_full[2], q_full[2], fin;
    uint64_t raw_full[kPmMaxStages], raw_empty[kPmMaxStages];
    UnitInfo unit[kPmMaxSlots], raw_unit[kPmMaxStages];
    alignas(16) float alpha[kPmRows], linv[kPmRows];
    // The plan: this CTA's first row tile and unit, its units, and for a row tile that
    // it begins, the CTAs that hold it (0: worked out from per and begin).
    long long warp_sum[16];
    uint2 warp_need[kPlanWarps];                      // CTAs, longest range of 32 row tiles
    long long total, per, begin;
    int first_tile, first_unit, first_units, count, parts;
    TileWalk first;                                   // of first_tile
    // The last part, written out by all warps.
    int last_tile, last_part;
    uint32_t tmem_base;
    volatile int abort;
};

template <bool kFp8, int kWidth>
struct PmSmem {
    static constexpr int kAtoms = kWidth / 64;
    static constexpr int kQAtoms = kAtoms - kPmQChannels / 64;      // of the queries, the others in tensor memory
    // Ring slots of one unit, as many as fit beside the stages of E4M3 units. Those are the
    // bytes in flight: four where HBM is to be kept busy, but with rotated channels only three
    // slots fit beside them, and the fourth slot is worth more (33 requests behind 4100 tokens
    // 44.4 -> 40.8 us; without rotation 64 ragged requests 253 -> 270 us).
    static constexpr int kSlots = kFp8 ? 4 : (kWidth > DSA_KV_LORA ? 5 : 6);
    static constexpr int kStages = kWidth > DSA_KV_LORA ? 2 : 4;
    // Fetchers and wideners take alternate units. An even number of stages keeps a stage with
    // one of either; with an odd one, a stage's next fetch could come to wait for the release
    // of its second last unit before that of the last but two, which a parity cannot tell apart.
    static_assert(kStages % 2 == 0 && kStages <= kPmMaxStages, "stages");
    static constexpr uint32_t kQ = 0;                               // kQAtoms x [64 rows x 128 B]
    static constexpr uint32_t kKV = kQAtoms * kPmRows * 128;        // slots x kAtoms x [32 rows x 128 B]
    static constexpr uint32_t kSlot = kAtoms * kPmAtom;
    static constexpr uint32_t kP = kKV + kSlots * kSlot;
    static constexpr uint32_t kRaw = kP + kPmPBytes;                // stages x [32 rows x kWidth B]
    static constexpr uint32_t kStage = kPmTile * kWidth;
    static constexpr uint32_t kCtl = kRaw + (kFp8 ? kStages * kStage : 0);
    static constexpr int kBytes = (int)kCtl + (int)sizeof(PmCtl) + 1024;   // + alignment slack
};
static_assert(PmSmem<false, 576>::kBytes <= 232448 && PmSmem<false, 512>::kBytes <= 232448 &&
                  PmSmem<true, 576>::kBytes <= 232448 && PmSmem<true, 512>::kBytes <= 232448,
              "shared memory per block");
static_assert(PmSmem<false, 512>::kSlots <= kPmMaxSlots, "ring");
constexpr int kPmScratch = (65535 * 2 + pm_threads(false) - 1) / pm_threads(false) * 8;   // a sum a block of row tiles
static_assert(kPmScratch <= PmSmem<true, 512>::kSlot, "the plan's scratch");
static_assert(kPlanWarps * 32 <= pm_threads(false), "a thread a row tile");

// Bounded waits. pm_wait, of the issuers and the softmax, asks again as soon as the
// hardware answers. pm_sleep, of the loaders, gives it a hint to hold the warp until
// the phase completes: a dozen polling warps fill the queue to shared memory that
// every exchange, barrier and global store of the others goes through, but a warp on
// the path from scores to products loses more by waking late (the hint everywhere
// costs 3 to 9 %, nowhere 2 to 3 %).
DSA_DEVINL bool pm_try_sleep(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kPmSleepNs)
        : "memory");
    return ok != 0;
}

template <bool kSleep>
DSA_DEVINL bool pm_wait_as(PmCtl *ctl, uint64_t *bar, uint32_t parity) {
    auto done = [&]() { return kSleep ? pm_try_sleep(bar, parity) : mbar_try_wait(bar, parity); };
    if (done()) return true;
    const long long t0 = clock64();
    for (;;) {
        if (done()) return true;
        if (ctl->abort) return false;
        if (clock64() - t0 > kWaitLimitCycles) break;
    }
    raise_device_error(kErrWaitTimeout);
    ctl->abort = 1;
    return false;
}
DSA_DEVINL bool pm_wait(PmCtl *ctl, uint64_t *bar, uint32_t parity) { return pm_wait_as<false>(ctl, bar, parity); }
DSA_DEVINL bool pm_sleep(PmCtl *ctl, uint64_t *bar, uint32_t parity) { return pm_wait_as<true>(ctl, bar, parity); }

// Two probes whose answers are waited for together: bit i is set when barrier i's phase
// of the given parity has completed, for every lane of the warp.
DSA_DEVINL uint32_t pm_test2(uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 a, b;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
        "selp.u32 a, 1, 0, p;\n\tselp.u32 b, 2, 0, q;\n\tor.b32 %0, a, b;\n\t}"
        : "=r"(r)
        : "r"(smem_u32(bar0)), "r"(parity0), "r"(smem_u32(bar1)), "r"(parity1)
        : "memory");
    return __reduce_and_sync(0xffffffffu, r);
}

// One lane of a converged warp, chosen so that the compiler knows it is one:
// descriptors then stay in uniform registers (an `if (lane == 0)` costs about
// 155 cycles a tcgen05.mma, this about 30).
DSA_DEVINL bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Four E4M3 codes (low byte first) widened to bf16 pairs by integer moves and one
// multiplication: exponent and mantissa at bf16's places give the value times 2^-120,
// subnormals included, and the product with 2^120 is exact. A code in a 16-bit lane
// times 16 has them there and its sign 4 bits low: 240 times the sign bit moves it
// up. (Multiply-adds: shifts and logic would all fall on one pipe.) NaN codes
// (S.1111.111) would become 480: the result has bit 7 of their bytes set (adding 1
// to seven ones is the one sum that carries; other bits mean nothing).
DSA_DEVINL uint32_t e4m3x4_to_bf16x4(uint32_t v, uint32_t &lo, uint32_t &hi) {
    const uint32_t a = __byte_perm(v, 0, 0x4140), b = __byte_perm(v, 0, 0x4342);   // codes in low bytes
    uint32_t x, y;
    asm("mad.lo.u32 %0, %1, 240, %2;" : "=r"(x) : "r"(a & 0x00800080u), "r"(a * 16u));
    asm("mad.lo.u32 %0, %1, 240, %2;" : "=r"(y) : "r"(b & 0x00800080u), "r"(b * 16u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x7B807B80u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x7B807B80u));
    return (v & 0x7F7F7F7Fu) + 0x01010101u;
}

DSA_DEVINL unsigned warp_inclusive_sum(unsigned v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// The plan, worked out by every CTA from the lengths on the device, so that
// nothing depends on the host's bounds and ragged batches load every SM alike.
// The units of all row tiles in order are cut into equal ranges of `per` units,
// one a CTA; a row tile split over CTAs leaves partial results, of which a CTA
// then leaves at most two, one of its first and one of its last row tile. Where
// there are fewer row tiles than CTAs, whole CTAs are given to each instead if
// the longest range grows by less than a second part costs (its queries, its
// output: kPmPartUnits). scratch: shared, kPmScratch bytes of the ring's.
template <int kThreads>
DSA_DEVINL void pm_plan(PmCtl *ctl, void *scratch, const PrefixGeom &g, const RowTiles &rt, int P) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreads / 32;
    const int nb = (rt.count + kThreads - 1) / kThreads;
    constexpr int G = kPmGrid;
    TileWalk w;
    int units = 0;
    long long base = 0, total = 0, inc;
    int kb = 0;
    if (nb == 1) {
        if (tid < rt.count) {
            w.load(g, rt, tid, P);
            units = w.units;
        }
        inc = warp_inclusive_sum((unsigned)units, lane);   // fits: pm_sums_fit
        if (lane == 31) ctl->warp_sum[warp] = inc;
        if (tid == 0) ctl->count = ctl->parts = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            base += k < warp ? ctl->warp_sum[k] : 0;
            total += ctl->warp_sum[k];
        }
    } else {
        auto *block_sum = reinterpret_cast<long long *>(scratch);
        for (int k = tid; k < nb; k += kThreads) block_sum[k] = 0;
        if (tid == 0) ctl->count = ctl->parts = 0;
        __syncthreads();
        for (int k = 0; k < nb; ++k) {
            const int t = k * kThreads + tid;
            units = 0;
            if (t < rt.count) {
                w.load(g, rt, t, P);
                units = w.units;
            }
            long long s = units;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0 && s)
                atomicAdd(reinterpret_cast<unsigned long long *>(&block_sum[k]), (unsigned long long)s);
        }
        __syncthreads();
        for (int k = 0; k < nb; ++k) total += block_sum[k];
    }
    // a range shorter than kPmMinUnits is not worth its part; with more row tiles than
    // CTAs it is not the splitting that makes ranges short
    const long long per = max((total + G - 1) / G, (long long)(rt.count <= G ? kPmMinUnits : 1));
    const long long begin = per * blockIdx.x;
    if (tid == 0) {
        ctl->total = total;
        ctl->per = per;
        ctl->begin = begin;
    }
    if (rt.count > 1 && rt.count <= G && total < (1 << 24)) {
        // Thread t: 1 + floor(units (G - count) / total) CTAs for row tile t, no more than G
        // in all, and the longest range that they get. By reciprocals, short of the quotient
        // here and above it for the range. (By a thread a row tile: code that a CTA runs once
        // comes from memory, and one warp's unrolled loops over the row tiles took 1.3 us.)
        unsigned need = 0, each = 0;
        if (tid < rt.count) {
            const float share = (float)(G - rt.count) * rcp_approx((float)total) * (1.f - 0x1p-20f);
            need = 1u + (unsigned)((float)units * share);
            each = need == 1u ? (unsigned)units
                              : max((unsigned)((float)units * rcp_approx((float)need) * (1.f + 0x1p-20f)) + 1u,
                                    (unsigned)kPmMinUnits);
        }
        const unsigned inc_need = warp_inclusive_sum(need, lane);
        const unsigned longest_w = __reduce_max_sync(0xffffffffu, each);
        if (lane == 31 && warp < kPlanWarps) ctl->warp_need[warp] = make_uint2(inc_need, longest_w);
        __syncthreads();
        unsigned k = blockIdx.x - (inc_need - need), longest = 0;
#pragma unroll
        for (int i = 0; i < kPlanWarps; ++i) {
            const uint2 x = ctl->warp_need[i];
            k -= i < warp ? x.x : 0u;
            longest = max(longest, x.y);
        }
        if (longest < (unsigned)per + kPmPartUnits) {
            if (k < need) {
                const unsigned u = (unsigned)units, at = min(u, k * each);
                unsigned parts = (unsigned)((float)u * rcp_approx((float)each));
                while (parts * each < u) ++parts;
                while (parts > 1 && (parts - 1) * each >= u) --parts;
                ctl->first_tile = tid;
                ctl->first = w;
                ctl->first_unit = (int)at;
                ctl->first_units = units;
                ctl->count = (int)min(u - at, each);
                ctl->parts = (int)parts;
            }
            __syncthreads();
            return;
        }
    }
    if (begin < total) {
        if (nb > 1) {
            const auto *block_sum = reinterpret_cast<const long long *>(scratch);
            while (base + block_sum[kb] <= begin) base += block_sum[kb++];
            const int t = kb * kThreads + tid;
            units = 0;
            if (t < rt.count) {
                w.load(g, rt, t, P);
                units = w.units;
            }
            inc = warp_inclusive_sum((unsigned)units, lane);
            if (lane == 31) ctl->warp_sum[warp] = inc;
            __syncthreads();
            for (int k = 0; k < warp; ++k) base += ctl->warp_sum[k];
        }
        const long long first = base + inc - units;
        if (units > 0 && first <= begin && begin < first + units) {
            ctl->first_tile = kb * kThreads + tid;
            ctl->first = w;
            ctl->first_unit = (int)(begin - first);
            ctl->first_units = units;
            ctl->count = (int)min(per, total - begin);
        }
    }
    tc::fence_proxy_async_smem();                     // the scratch becomes the ring
    __syncthreads();
}

// One of the eight pieces (128-channel block blk / 2, 32-row half blk % 2) of O^T in a
// lane quarter, out of tensor memory. A part's fp32 rows: lane l holds channel l of 32
// rows, and 32 lanes write 128 bytes of a row. Normalised bf16 rows: the fragment shape
// gives a thread two rows of one channel, the transposing store makes rows of 32 channels
// of them in shared memory (2 KB at `stage`, 16-byte columns exclusive-or'ed with the
// row pair), and 16-byte pieces go out: 12 accesses a piece where exchanging channels
// between lanes took 40.
DSA_DEVINL void pm_write_rows(const PmCtl *ctl, uint32_t tquarter, int quarter, int blk, int nr, size_t row0,
                              int part_slot, uint32_t stage, __nv_bfloat16 *out, float *part) {
    const int lane = threadIdx.x & 31;
    const int r0 = (blk & 1) * 32, L = (blk >> 1) * 128 + 32 * quarter;
    const uint32_t src = tquarter + (blk >> 1) * 64 + (blk & 1) * 32;
    if (r0 >= nr) return;
    if (part_slot >= 0) {
        uint32_t o[32];
        tc::tmem_ld32(src, o);
        tc::tmem_wait_ld();
        float *po = part + ((size_t)part_slot * kPmRows + r0) * kL + L + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (r0 + j < nr) po[(size_t)j * kL] = __uint_as_float(o[j]);
        return;
    }
    // Registers 4g .. 4g+3 of each half: channels lane/4 and lane/4 + 8, rows
    // 8g + 2 (lane%4) and the next.
    uint32_t a[16], b[16];
    tc::tmem_ld16x256b_x4(src, a);
    tc::tmem_ld16x256b_x4(src + (16u << 16), b);
    tc::tmem_wait_ld();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const float2 f = *reinterpret_cast<const float2 *>(&ctl->linv[r0 + 8 * g + 2 * (lane & 3)]);
        // a row that saw nothing is 0 whatever its column holds
        auto pack = [&](uint32_t x, uint32_t y) {
            return pack_bf16x2(f.x != 0.f ? __uint_as_float(x) * f.x : 0.f,
                               f.y != 0.f ? __uint_as_float(y) * f.y : 0.f);
        };
        const int r = 8 * g + (lane & 7);
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         stage + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4)),
                     "r"(pack(a[4 * g], a[4 * g + 1])), "r"(pack(a[4 * g + 2], a[4 * g + 3])),
                     "r"(pack(b[4 * g], b[4 * g + 1])), "r"(pack(b[4 * g + 2], b[4 * g + 3]))
                     : "memory");
    }
    __syncwarp();
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "r"(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4))
                     : "memory");
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 8 * i + (lane >> 2);
        if (r < nr) *reinterpret_cast<uint4 *>(out + (row0 + r) * kL + L + 8 * (lane & 3)) = v[i];
    }
    __syncwarp();                                     // the next piece takes the same stage
}

// kv: kv_rows rows of kWidth bf16, or E4M3 bytes (kFp8; widened to bf16, which
// is exact). box_rows: rows of a box of kv_map, 0 where pages allow none.
template <bool kFp8, int kWidth>
__global__ void __launch_bounds__(pm_threads(kFp8), 1)
prefix_mla_kernel(const __grid_constant__ CUtensorMap kv_map, int box_rows,
                  const __nv_bfloat16 *__restrict__ q, const void *__restrict__ kv,
                  const PrefixGeom g, int Hm, float scale_log2, float out_scale,
                  float *__restrict__ part, float2 *__restrict__ part_ml,
                  MergeEntry *__restrict__ merge, __nv_bfloat16 *__restrict__ out,
                  float *__restrict__ lse) {
    using S = PmSmem<kFp8, kWidth>;
    constexpr int kAtoms = S::kAtoms, kPmSlots = S::kSlots, kPmStages = S::kStages;
    extern __shared__ uint8_t pm_smem_raw[];
    const uint32_t raw = smem_u32(pm_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;           // 128B-swizzle atoms need 1 KB
    uint8_t *gbase = pm_smem_raw + (base - raw);
    PmCtl *ctl = reinterpret_cast<PmCtl *>(gbase + S::kCtl);
    const uint32_t sQ = base + S::kQ, sKV = base + S::kKV, sP = base + S::kP;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const RowTiles rt(g.Q, Hm);

    if (warp == kPmIssuer) {
        tc::tmem_alloc(&ctl->tmem_base, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < kPmSlots; ++i) {
            // four warps: a word from each, and where lanes copy rows, every lane's copies
            mbar_init(&ctl->kv_full[i], kFp8 ? 4 : 4 * 32 + 4);
            mbar_init(&ctl->kv_empty[i], 1);
        }
        for (int i = 0; i < kPmSBufs; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->s_empty[i], 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->p_full[i], 128);
        }
        for (int i = 0; i < kPmStages; ++i) {
            mbar_init(&ctl->raw_full[i], 1);
            mbar_init(&ctl->raw_empty[i], 4);
        }
        mbar_init(&ctl->q_full[0], 128);
        mbar_init(&ctl->q_full[1], 128);
        mbar_init(&ctl->fin, kFp8 ? 2 : 3);       // a commit of every issuer
        ctl->abort = 0;
        ctl->last_tile = -1;
        fence_mbarrier_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
    if (!kFp8 && box_rows > 0 && tid == 32)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kv_map)));
    // Page tables and queries towards L2, each CTA its share, while the plan is worked out
    // (a hint reads nothing: what a predecessor still writes is written to L2).
    {
        const long long at = ((long long)tid * gridDim.x + blockIdx.x) * 128;
        const long long q_bytes = (long long)rt.total_rows * kWidth * 2;
        if (at < q_bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(q) + at));
        if (at < (long long)g.B * g.max_blocks * 4)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(g.block_table) + at));
        if (at < (long long)g.prefix_blocks * 4)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(g.prefix_table) + at));
    }
    pdl_wait();                       // queries, lengths and cache rows may come from the predecessor
    pdl_launch_dependents();

    const int P = g.shared_len();
    pm_plan<pm_threads(kFp8)>(ctl, gbase + S::kKV, g, rt, P);
    const int n = ctl->count;
    const bool by_tile = rt.count <= kPmGrid;
    if (!by_tile && tid == 0) {
        // merge entries by CTA: the second CTA of a split row tile holds it
        MergeEntry e{-1, 0, 0, 0};
        if (n > 0 && ctl->first_unit > 0) {
            const long long tb = ctl->begin - ctl->first_unit;
            const int cf = (int)(tb / ctl->per), cl = (int)((tb + ctl->first_units - 1) / ctl->per);
            if (cf == (int)blockIdx.x - 1) e = MergeEntry{ctl->first_tile, cf, cl - cf + 1, 0};
        }
        merge[blockIdx.x] = e;
    }

    if (warp == kPmIssuer || (!kFp8 && warp == kPmIssuer + 2)) {
        // ------------------------------------------------------------------ S issuers
        // S(c)[64 rows x 32 tokens] = Q K^T, kWidth / 16 K-steps, up to two units
        // ahead of PV. While the tensor cores read their operands an access to shared memory
        // takes over 100 cycles: two waits and the unit's word take an issuer 650 of 1290
        // cycles a unit. bf16 therefore has two of them, for even and for odd units (64
        // requests behind 16384 tokens 387 -> 372 us, 64 of two queries behind 16389 112 ->
        // 108 us; one row of 512 11.8 -> 12.3 us); E4M3 does better with the warp as a second
        // fetcher (64 ragged requests 262 us, with one fetcher and two issuers 292 us).
        constexpr uint32_t idS = tc::idesc_bf16(64, kPmTile, false, false);
        const uint64_t a0 = tc::desc_sw128(sQ, 16, 1024);
        constexpr int kStep = kFp8 ? 1 : 2;
        bool ok = true;
        uint32_t seen = 4u;                               // part of this warp's last unit
        for (int c = (warp - kPmIssuer) >> 1; c < n; c += kStep) {
            const int slot = c % kPmSlots, sb = c & 1;
            const uint32_t d = tmem + kPmSCol + (uint32_t)(sb * kPmTile);
            ok = pm_wait(ctl, &ctl->kv_full[slot], (c / kPmSlots) & 1);
            const uint32_t word = ctl->unit[slot].word, part = word / kUnitPart & 3u;
            if (ok && c >= 2) ok = pm_wait(ctl, &ctl->s_empty[sb], ((c >> 1) - 1) & 1);
            // Parts alternate two barriers: a part whose only unit went to the other warp
            // passes unseen here, and its barrier then does not stand for the next one's.
            if (ok && part != seen) ok = pm_wait(ctl, &ctl->q_full[part & 1], part >> 1);
            seen = part;
            if (!__all_sync(0xffffffffu, ok)) break;
            tc::fence_after_sync();
            if (word & kUnitCopied) tc::fence_proxy_async_smem();   // cp.async writes, tensor-core reads
            if (elect_one()) {
                const uint64_t b0 = tc::desc_sw128(sKV + slot * S::kSlot, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < kPmQSteps; ++kk)
                    tc::mma_bf16_ts(d, tmem + kPmQCol + kk * 8,
                                    b0 + (uint64_t)(((kk >> 2) * kPmAtom + (kk & 3) * 32) >> 4), idS,
                                    kk > 0 ? 1u : 0u);
#pragma unroll
                for (int kk = kPmQSteps; kk < kWidth / 16; ++kk) {
                    const int ka = kk - kPmQSteps;
                    tc::mma_bf16_ss(d, a0 + (uint64_t)(((ka >> 2) * kPmRows * 128 + (ka & 3) * 32) >> 4),
                                    b0 + (uint64_t)(((kk >> 2) * kPmAtom + (kk & 3) * 32) >> 4), idS, 1u);
                }
                tc::mma_commit(&ctl->s_full[sb]);
            }
            __syncwarp();
        }
        __syncwarp();
        if (elect_one()) tc::mma_commit(&ctl->fin);
        __syncwarp();
    } else if (warp == kPmIssuer + 1) {
        // ------------------------------------------------------------------ PV issuer
        // PV(c): O^T[128 b .. + 127][the unit's rows] += V^T P^T for the four
        // 128-channel blocks b. Rows are the N dimension of PV, so a unit that one
        // query sees touches that query's columns alone (a NaN among its values
        // reaches no other).
        bool ok = true;
        int slot = 0;
        for (int c = 0; c < n; ++c) {
            const int pb = c & 1;
            ok = pm_wait(ctl, &ctl->kv_full[slot], (c / kPmSlots) & 1);
            const uint32_t word = __shfl_sync(0xffffffffu, ctl->unit[slot].word, 0);
            const uint32_t row0 = word & 255u;
            const uint32_t id = tc::idesc_bf16(128, 0, true, false) | (((word >> 8) & 255u) >> 3 << 17);
            // V^T: MN-major, 64-channel atoms kPmAtom apart, 8-token groups 1 KB apart
            const uint64_t a0 = tc::desc_sw128(sKV + slot * S::kSlot, kPmAtom, 1024);
            // P^T: K-major, 128-byte rows (this buffer's half), 8-row groups 1 KB apart
            const uint64_t b0 = tc::desc_sw128(sP + row0 * 128 + pb * 64, 16, 1024);
            if (word & kUnitCopied) tc::fence_proxy_async_smem();   // cp.async writes, tensor-core reads
            if (ok) ok = pm_wait(ctl, &ctl->p_full[pb], (c >> 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kPmTile / 16; ++ks)
#pragma unroll
                    for (int blk = 0; blk < 4; ++blk)
                        tc::mma_bf16_ss(tmem + (uint32_t)(blk * kPmRows) + row0,
                                        a0 + (uint64_t)((blk * 2 * kPmAtom + ks * 2048) >> 4),
                                        b0 + (uint64_t)((ks * 32) >> 4), id,
                                        (ks > 0 || !(word & kUnitFresh)) ? 1u : 0u);
                tc::mma_commit(&ctl->kv_empty[slot]);
            }
            __syncwarp();
            if (++slot == kPmSlots) slot = 0;
        }
        __syncwarp();
        if (elect_one()) tc::mma_commit(&ctl->fin);
        __syncwarp();
    } else if (kFp8 && warp >= 4 && warp < 12) {
        // ------------------------------------------------------------------ widening (E4M3, warps 4-11)
        // Two groups of four warps take alternate units from the stages, widen them to
        // bf16 exactly, eight rows a warp, and store them into the swizzled slots; rows
        // where there is no token become zeros. Eight codes make one 16-byte column of a
        // slot's row: lane l takes columns l and l + 32, so that neither access conflicts.
        const int sub = (warp - 4) & 3;
        constexpr int kCols = kWidth / 8, kLoads = 8 * kCols / 32;         // 16 or 18 a lane
        for (int c = (warp - 4) >> 2; c < n; c += 2) {
            const int slot = c % kPmSlots, stage = c % kPmStages;
            bool ok = pm_sleep(ctl, &ctl->raw_full[stage], (c / kPmStages) & 1);
            const UnitInfo info = ctl->raw_unit[stage];
            const uint8_t *src = gbase + S::kRaw + stage * S::kStage;
            const uint32_t dst0 = sKV + slot * S::kSlot;
            // columns l and l + 32 of row i, then columns 64 .. 71 of four rows a time
            auto row_of = [&](int i) { return 8 * sub + (i < 16 ? i >> 1 : 4 * (i - 16) + (lane >> 3)); };
            auto col_of = [&](int i) { return i < 16 ? lane + 32 * (i & 1) : 64 + (lane & 7); };
            uint2 x[kLoads];
            uint32_t nan = 0;                         // bit 7 of every byte: a NaN code was there
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = row_of(i);
                x[i] = (info.valid >> r) & 1u ? *reinterpret_cast<const uint2 *>(src + r * kWidth + 8 * col_of(i))
                                              : make_uint2(0u, 0u);
            }
            // Now the codes are in registers. Two stages are released here, so that the next
            // copies run behind the widening (4 requests of 131072 tokens with rope 145 -> 129
            // us); of four it only puts the loads' latency before the wait for the slot (64
            // ragged requests 258 -> 271 us).
            constexpr bool kEarly = kPmStages == 2;
            if constexpr (kEarly) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->raw_empty[stage]);
            }
            if (ok && c >= kPmSlots) ok = pm_sleep(ctl, &ctl->kv_empty[slot], ((c / kPmSlots) - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            auto store = [&](int i, const uint32_t (&w)[4]) {
                const int r = row_of(i), cc = col_of(i);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 dst0 + (cc >> 3) * kPmAtom + r * 128 + (((cc & 7) ^ (r & 7)) << 4)),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
            };
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                uint32_t w[4];
                nan |= e4m3x4_to_bf16x4(x[i].x, w[0], w[1]);
                nan |= e4m3x4_to_bf16x4(x[i].y, w[2], w[3]);
                store(i, w);
            }
            if (nan & 0x80808080u) {
                // some code of this lane was NaN: its columns again by the conversion instruction
                auto again = [&](int i, uint2 v) {
                    const uint32_t w[4] = {e4m3x2_to_bf16x2((uint16_t)(v.x & 0xFFFFu)),
                                           e4m3x2_to_bf16x2((uint16_t)(v.x >> 16)),
                                           e4m3x2_to_bf16x2((uint16_t)(v.y & 0xFFFFu)),
                                           e4m3x2_to_bf16x2((uint16_t)(v.y >> 16))};
                    store(i, w);
                };
                if constexpr (kEarly) {
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) again(i, x[i]);
                } else {
                    // out of the stage: the codes need not stay in registers (4 % on all)
#pragma unroll 1
                    for (int i = 0; i < kLoads; ++i)
                        if ((info.valid >> row_of(i)) & 1u)
                            again(i, *reinterpret_cast<const uint2 *>(src + row_of(i) * kWidth + 8 * col_of(i)));
                }
            }
            tc::fence_proxy_async_smem();               // generic stores -> tensor-core reads
            __syncwarp();
            if (lane == 0) {
                if (sub == 0) ctl->unit[slot] = info;
                mbar_arrive(&ctl->kv_full[slot]);
                if (!kEarly) mbar_arrive(&ctl->raw_empty[stage]);
            }
            __syncwarp();
        }
    } else if (kFp8 ? warp >= kPmIssuer + 2 : warp >= 4 && warp < 12) {
        // ------------------------------------------------------------------ loaders
        // bf16: two groups of four warps fill alternate units of the ring; E4M3: two
        // warps fill alternate stages. Lane l of every warp finds
        // the cache row of the unit's token l. Where the 32 rows are whole boxes of
        // the tensor map (pages that are a multiple of 16 rows, away from the ends
        // of a segment) one thread brings them by TMA; else warp i of the group
        // copies rows 8i .. 8i+7 in 16-byte pieces, zero-filled where there is no
        // token: what lies behind a sequence may hold anything, and a weight of 0
        // times a NaN would not be 0.
        const int grp = kFp8 ? warp - kPmIssuer - 2 : (warp - 4) >> 2, sub = kFp8 ? 0 : (warp - 4) & 3;
        TileWalk w;
        int tile = n > 0 ? ctl->first_tile : 0, u = n > 0 ? ctl->first_unit : 0;
        int part_begin = u;                               // the part's first unit in its tile
        const int tile0 = tile;
        if (n > 0) w = ctl->first;
        long long global_unit = ctl->begin;
        int left = n;                                     // units from the current one on
        // The segment of the current unit (-1: the prefix), its tokens s0 .. s1-1, the unit's
        // first token, the units from this one to the segment's end, whether the unit is the
        // segment's first, the queries whose common units this part has had; and for the row
        // lookups the request's table.
        int seg = -1, s0 = 0, s1 = 0, tok0 = 0, seg_left = 0, met = 0;
        bool seg_first = false;
        uint32_t rows_word = 0;
        const int32_t *pages = nullptr;
        // the unit `skip` units behind the start of segment j of the tile, or of a later one
        auto enter_segment = [&](int j, int skip) {
            if (rt.qpt == 1) {                            // one query: its whole sequence
                seg = 1;
                seg_first = skip == 0;
                s1 = w.vis[0];
                seg_left = w.units - skip;
                tok0 = skip * kPmTile;
                pages = g.block_table + (size_t)(w.active ? w.req[0] : 0) * g.max_blocks;
                rows_word = ((uint32_t)kPmRows << 8) | ((uint32_t)w.active << 24);
                return;
            }
            for (;; ++j) {
                int nu = j < 0 ? w.npre : 0;
#pragma unroll
                for (int i = 0; i < 2 * kPmQueries; ++i)
                    if (j == i) nu = w.segment_units(i, P);
                if (skip < nu || j >= 2 * kPmQueries) {
                    seg_left = nu - skip;
                    break;
                }
                skip -= nu;
            }
            const int k = j >> 1;
            const bool common = j >= 0 && !(j & 1);
            seg = j;
            seg_first = skip == 0;
            s0 = j >= 0 && w.shared ? P : 0;
            s1 = j < 0 ? P : 0;
            int b = 0, run = 1;
#pragma unroll
            for (int i = 0; i < kPmQueries; ++i)
                if (j >= 0 && k == i) {
                    s1 = common ? w.common[i] : w.vis[i];
                    if (!common) s0 = max(s0, w.common[i]);
                    b = w.req[i];
                    run = common ? w.run(i) : 1;
                }
            if (common) met |= ((1 << run) - 1) << k;
            if (w.active == 0) { s1 = 0; b = 0; seg_left = 1; }   // no query sees a token: an empty unit
            pages = g.block_table + (size_t)b * g.max_blocks;
            tok0 = (int)((unsigned)s0 / kPmTile * kPmTile) + skip * kPmTile;
            rows_word = (j < 0 || rt.qpt == 1 || w.active == 0 ? (uint32_t)kPmRows << 8
                                                              : (uint32_t)(k * Hm) | ((uint32_t)(run * Hm) << 8)) |
                        ((uint32_t)w.active << 24);
        };
        // describe the current unit; returns the row of this lane's token
        auto describe = [&](UnitInfo &info) -> int {
            const bool first = u == part_begin, last = left == 1 || u + 1 == w.units;
            const bool summed = (w.shared && part_begin < w.npre) || ((seg & 1) && ((met >> (seg >> 1)) & 1));
            const bool fresh = first || (seg >= 0 && seg_first && !summed);
            info.word = rows_word | (first ? kUnitFirst : 0u) | (last ? kUnitLast : 0u) | (fresh ? kUnitFresh : 0u) |
                        (uint32_t)((tile - tile0) & 3) * kUnitPart;
            // read on the last unit alone: a part that is the whole tile has no slot
            info.part = part_begin == 0 && u + 1 == w.units ? -1 : 2 * (int)blockIdx.x + (part_begin == 0 ? 1 : 0);
            const int t = tok0 + lane;
            return t >= s0 && t < s1 ? g.row(pages, t, P) : -1;
        };
        // merge entries by row tile, left by the CTA that begins it
        auto enter_tile = [&](int t, long long begin, int units) {
            if (by_tile && grp == 0 && sub == 0 && lane == 0) {
                const int parts = ctl->parts ? ctl->parts
                                             : (int)((begin + units - 1) / ctl->per) - (int)blockIdx.x + 1;
                merge[t] = MergeEntry{t, (int)blockIdx.x, parts, 0};
            }
        };
        // one unit forward; false behind the last
        auto advance = [&]() -> bool {
            if (--left <= 0) return false;
            ++global_unit;
            ++u;
            tok0 += kPmTile;
            seg_first = false;
            if (--seg_left > 0) return true;
            if (u >= w.units) {
                u = 0;
                part_begin = 0;
                met = 0;
                w.load(g, rt, ++tile, P);
                enter_tile(tile, global_unit, w.units);
                enter_segment(w.npre > 0 ? -1 : 0, 0);
            } else {
                enter_segment(seg + 1, 0);
            }
            return true;
        };

        if (n > 0) enter_segment(w.npre > 0 ? -1 : 0, u);
        const bool begins = n > 0 && u == 0;              // its entry is written behind the first copies
        bool more = n > 0;
        if (grp == 1) more = more && advance();
        int slot = grp;
        uint32_t ph = 1;                                  // parity of the slot's last release
        auto next_slot = [&]() {
            slot += 2;
            if (slot >= kPmSlots) { slot -= kPmSlots; ph ^= 1u; }
        };
        UnitInfo info;
        int row = -1;
        if (more) row = describe(info);
        int c = grp;                                      // behind the loop: the first unit not copied
        if constexpr (!kFp8) {
            for (; more; c += 2, next_slot()) {
                const uint32_t dst0 = sKV + slot * S::kSlot;
                const bool ok = c < kPmSlots || pm_sleep(ctl, &ctl->kv_empty[slot], ph);
                if (!__all_sync(0xffffffffu, ok)) break;
                info.valid = __ballot_sync(0xffffffffu, row >= 0);
                bool boxes = box_rows > 0 && info.valid == 0xffffffffu;
                if (boxes) {
                    const int first = __shfl_sync(0xffffffffu, row, lane & ~(box_rows - 1));
                    boxes = __all_sync(0xffffffffu, row == first + (lane & (box_rows - 1)));
                }
                if (boxes) {
                    const int row_b = __shfl_sync(0xffffffffu, row, box_rows & 31);   // the second box
                    const int row_a = __shfl_sync(0xffffffffu, row, 0);
                    if (sub == 0) {
                        if (elect_one()) {
                            ctl->unit[slot] = info;
                            mbar_arrive_expect_tx(&ctl->kv_full[slot], kPmTile * kWidth * 2);
                            if (box_rows == kPmTile) {
                                tma_load_3d(dst0, &kv_map, 0, row_a, 0, &ctl->kv_full[slot]);
                            } else {
#pragma unroll
                                for (int a = 0; a < kAtoms; ++a) {
                                    tma_load_3d(dst0 + a * kPmAtom, &kv_map, 0, row_a, a, &ctl->kv_full[slot]);
                                    tma_load_3d(dst0 + a * kPmAtom + 16 * 128, &kv_map, 0, row_b, a,
                                                &ctl->kv_full[slot]);
                                }
                            }
                        }
                    } else if (lane == 0) {
                        mbar_arrive(&ctl->kv_full[slot]);
                    }
                    __syncwarp();
                    mbar_arrive(&ctl->kv_full[slot]);
                } else {
                    const auto *kvb = reinterpret_cast<const __nv_bfloat16 *>(kv);
#pragma unroll
                    for (int rr = 0; rr < 8; ++rr) {
                        const int r = 8 * sub + rr;
                        const int src_row = __shfl_sync(0xffffffffu, row, r);
                        const __nv_bfloat16 *src = src_row >= 0 ? kvb + (size_t)src_row * kWidth : q;   // q: never read
                        const uint32_t nb = src_row >= 0 ? 16u : 0u;
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int cc = lane + 32 * hh;                    // 16-byte piece of the row
                            tc::cp_async16_zfill(dst0 + (cc >> 3) * kPmAtom + r * 128 + (((cc & 7) ^ (r & 7)) << 4),
                                                 src_row >= 0 ? src + cc * 8 : src, nb);
                        }
                    }
                    if constexpr (kWidth > DSA_KV_LORA) {
                        // the rotated channels: eight pieces a row, four rows a pass
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            const int r = 8 * sub + 4 * rr + (lane >> 3), cc = lane & 7;
                            const int src_row = __shfl_sync(0xffffffffu, row, r);
                            const __nv_bfloat16 *src =
                                src_row >= 0 ? kvb + (size_t)src_row * kWidth + DSA_KV_LORA + cc * 8 : q;
                            tc::cp_async16_zfill(dst0 + (kAtoms - 1) * kPmAtom + r * 128 + ((cc ^ (r & 7)) << 4),
                                                 src, src_row >= 0 ? 16u : 0u);
                        }
                    }
                    if (lane == 0) {
                        info.word |= kUnitCopied;
                        if (sub == 0) ctl->unit[slot] = info;
                        mbar_arrive(&ctl->kv_full[slot]);
                    }
                    tc::cp_async_arrive_noinc(&ctl->kv_full[slot]);
                }
                more = advance() && advance();
                if (more) row = describe(info);           // its page lookups run behind this unit's copies
            }
        } else {
            // A bulk copy for every run of rows that lie one after the other: one for a unit
            // within a page, up to three with pages of 16 or more rows of any number.
            const auto *kv8 = reinterpret_cast<const uint8_t *>(kv);
            for (; more; c += 2) {
                const int stage = c % kPmStages;
                const bool ok = c < kPmStages || pm_sleep(ctl, &ctl->raw_empty[stage], ((c / kPmStages) - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                info.valid = __ballot_sync(0xffffffffu, row >= 0);
                const int prev = __shfl_up_sync(0xffffffffu, row, 1);
                const bool begins_run = row >= 0 && (lane == 0 || prev < 0 || row != prev + 1);
                // the lanes that end a run before them
                const uint32_t ends = __ballot_sync(0xffffffffu, begins_run || row < 0) & (0xfffffffeu << lane);
                uint8_t *dst = gbase + S::kRaw + stage * S::kStage;
                if (elect_one()) {
                    ctl->raw_unit[stage] = info;
                    mbar_arrive_expect_tx(&ctl->raw_full[stage], __popc(info.valid) * kWidth);
                }
                __syncwarp();
                if (begins_run)
                    bulk_g2s(dst + lane * kWidth, kv8 + (size_t)row * kWidth, ((ends ? __ffs(ends) - 1 : 32) - lane) * kWidth,
                             &ctl->raw_full[stage]);
                __syncwarp();
                more = advance() && advance();
                if (more) row = describe(info);
            }
        }
        if (ctl->abort && sub == 0) {
            // A wait ran out: the bulk copies under way land before the block leaves its shared
            // memory. (A slot's earlier unit was released before its next one was copied.)
            constexpr int kRing = kFp8 ? kPmStages : kPmSlots;
            for (int k = c - 2; k >= 0 && k > c - 2 - kRing; k -= 2)
                (void)mbar_wait(kFp8 ? &ctl->raw_full[k % kRing] : &ctl->kv_full[k % kRing], (k / kRing) & 1);
        }
        if (begins) enter_tile(ctl->first_tile, ctl->begin, ctl->first_units);
        tc::cp_async_wait_all();          // nothing of this warp in flight past here
    } else if (warp < 4) {
        // ------------------------------------------------------------------ softmax (warps 0-3)
        // S is read with the 16x64b tensor-memory shape: thread t of warp wq holds
        // row hh = 16 wq + (t>>2) + 8 (t&1) and the unit's tokens of parity
        // par = (t>>1)&1; its partner t^2 holds the other parity of the same row.
        const int wq = warp, wtid = tid;
        const int hh = 16 * wq + (lane >> 2) + 8 * (lane & 1);
        const int par = (lane >> 1) & 1;
        const bool owner = par == 0;          // writes the row's values
        const uint32_t tl = tmem + ((uint32_t)(32 * wq) << 16);
        const int hq = rt.qpt > 1 ? hh / Hm : 0;   // the row's query within its tile
        float m_used = -INFINITY, l = 0.f;
        bool failed = false;

        // The queries of a row tile: channels from 384 on into shared memory (swizzled,
        // K-major), the others into tensor memory, where this thread's row hh has its
        // pairs of channels as columns: thread and partner load alternate 16-byte
        // vectors (four columns) and swap the columns of the other's parity.
        auto load_q = [&](int tile, auto batch) {
            const int row0 = rt.first_row(tile), nr = rt.rows(tile);
            constexpr int kPieces = S::kQAtoms * 8;
#pragma unroll 2
            for (int x = wtid; x < kPmRows * kPieces; x += 128) {
                const int r = x / kPieces, cc = x % kPieces;
                const uint32_t dst = sQ + (cc >> 3) * (kPmRows * 128) + r * 128 + (((cc & 7) ^ (r & 7)) << 4);
                if (r < nr)
                    tc::cp_async16(dst, q + (size_t)(row0 + r) * kWidth + kPmQChannels + cc * 8);
                else
                    tc::st_shared_zero16(dst);
            }
            const uint4 *src = reinterpret_cast<const uint4 *>(q + (size_t)(row0 + min(hh, nr - 1)) * kWidth) + par;
            // Batches of 32-column blocks, a batch's loads in flight at once: the first row
            // tile's are what a CTA waits for, a later one's hide behind its last PV and have
            // fewer registers (two batches in flight spill there).
            constexpr int kBlocks = kPmQSteps * 8 / 32, kBatch = decltype(batch)::value;
            static_assert(kBlocks % kBatch == 0, "whole batches");
#pragma unroll
            for (int b0 = 0; b0 < kBlocks; b0 += kBatch) {
                uint4 x[kBatch][4];
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[b][i] = src[(b0 + b) * 8 + 2 * i];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // columns 8i + 4 par .. + 3 of the block are here; keep those of parity par
                        const uint32_t s0 = par ? x[b][i].x : x[b][i].y, s1 = par ? x[b][i].z : x[b][i].w;
                        const uint32_t k0 = par ? x[b][i].y : x[b][i].x, k1 = par ? x[b][i].w : x[b][i].z;
                        const uint32_t g0 = __shfl_xor_sync(0xffffffffu, s0, 2);
                        const uint32_t g1 = __shfl_xor_sync(0xffffffffu, s1, 2);
                        // register j is column par + 2j
                        o[4 * i + 0] = par ? g0 : k0;
                        o[4 * i + 1] = par ? g1 : k1;
                        o[4 * i + 2] = par ? k0 : g0;
                        o[4 * i + 3] = par ? k1 : g1;
                    }
                    if (hh >= nr)
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = 0u;
                    tc::tmem_st16x64b_x16(tl + kPmQCol + (uint32_t)((b0 + b) * 32), o);
                }
            }
            tc::tmem_wait_st();
        };
        auto release_q = [&](int tile) {
            tc::cp_async_wait_all();
            tc::fence_proxy_async_smem();
            tc::fence_before_sync();
            mbar_arrive(&ctl->q_full[(tile - ctl->first_tile) & 1]);
        };
        int tile = n > 0 ? ctl->first_tile : 0;       // a CTA's parts are consecutive row tiles
        if (n > 0) {
            load_q(tile, std::integral_constant<int, 3>{});
            release_q(tile);
        }
        // Ring positions and parities of units c, c - 1 and c - 2 (a PV frees its slot,
        // and has then read its P buffer).
        int slot = 0, slot1 = 0, slot2 = 0;
        uint32_t par0 = 0, par1 = 0, par2 = 0;
        UnitInfo info = {};
        if (n > 0) {
            (void)pm_wait(ctl, &ctl->kv_full[0], 0);
            info = ctl->unit[0];
        }
        for (int c = 0; c < n; ++c) {
            const int pb = c & 1, sb = c % kPmSBufs;
            const int nslot = slot + 1 == kPmSlots ? 0 : slot + 1;
            const uint32_t npar = nslot == 0 ? par0 ^ 1u : par0;
            bool bad = !pm_wait(ctl, &ctl->s_full[sb], (c / kPmSBufs) & 1);
            tc::fence_after_sync();
            uint32_t sr[16];                              // tokens par + 2i
            tc::tmem_ld16x64b_x16(tl + kPmSCol + (uint32_t)(sb * kPmTile), sr);
            // What the end of this turn needs, asked for while the scores arrive: shared
            // memory answers slowly while the tensor cores read their operands.
            const uint32_t ready = pm_test2(&ctl->kv_full[nslot], npar, &ctl->kv_empty[slot2], par2);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            mbar_arrive(&ctl->s_empty[sb]);
            UnitInfo next = ctl->unit[nslot];             // the next unit's once it is ready

            const bool mine = (uint32_t)hh - info.row0() < info.rows() && ((info.word >> (24 + hq)) & 1u);
            const uint32_t vm = mine ? info.valid >> par : 0u;
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = __uint_as_float(sr[i]) * scale_log2;
            if ((vm & 0x55555555u) != 0x55555555u) {
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = ((vm >> (2 * i)) & 1) ? z[i] : -INFINITY;
            }
            float m4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmaxf(fmaxf(z[i], z[i + 4]), fmaxf(z[i + 8], z[i + 12]));
            float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            float alpha = 1.f;
            bool moved = false;
            if (mx > m_used + kLazyRescale) {
                // nothing summed before: nothing to rescale
                moved = m_used != -INFINITY && !info.is(kUnitFirst);
                alpha = ex2(m_used - mx);
                m_used = mx;
            }
            // a row without a token so far: its weights are 0 (z = -inf) and not NaN
            const float m_ref = m_used == -INFINITY ? 0.f : m_used;
            float p4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                z[i] = ex2(z[i] - m_ref);
                p4[i & 3] += z[i];   // fp32 weights: the row sum and lse stay exact to fp32
            }
            float psum = (p4[0] + p4[1]) + (p4[2] + p4[3]);
            psum += __shfl_xor_sync(0xffffffffu, psum, 2);
            l = fmaf(l, alpha, psum);
            // bf16 P row: this thread packs tokens 16 par .. 16 par + 15, taking the
            // other parity from its partner.
            uint32_t pk[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float recv = __shfl_xor_sync(0xffffffffu, par ? z[k] : z[k + 8], 2);
                pk[k] = par ? pack_bf16x2(recv, z[k + 8]) : pack_bf16x2(z[k], recv);
            }
            if (c >= 2 && !(ready & 2u)) bad = bad || !pm_wait(ctl, &ctl->kv_empty[slot2], par2);
            // One barrier a unit; a second only when some row rescales or a wait failed.
            const bool need = tc::named_bar_or(2, 128, bad || moved);
            if (need) {
                if (owner) ctl->alpha[hh] = alpha;
                if (tc::named_bar_or(2, 128, bad)) { failed = true; break; }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c16 = 4 * pb + 2 * par + k;     // 16-byte piece of the 128-byte row
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 sP + hh * 128 + ((c16 ^ (hh & 7)) << 4)),
                             "r"(pk[4 * k]), "r"(pk[4 * k + 1]), "r"(pk[4 * k + 2]), "r"(pk[4 * k + 3])
                             : "memory");
            }
            if (need) {
                // O^T columns of rescaled rows times alpha, after PV(c-1) has landed
                bad = !pm_wait(ctl, &ctl->kv_empty[slot1], par1);
                if (tc::named_bar_or(2, 128, bad)) { failed = true; break; }
                tc::fence_after_sync();
#pragma unroll 1
                for (int blk = 0; blk < 8; ++blk) {
                    uint32_t o[32];
                    const uint32_t ta = tl + (blk >> 1) * 64 + (blk & 1) * 32;
                    tc::tmem_ld32(ta, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&ctl->alpha[(blk & 1) * 32 + j]);
                        o[j] = __float_as_uint(__uint_as_float(o[j]) * f.x);
                        o[j + 1] = __float_as_uint(__uint_as_float(o[j + 1]) * f.y);
                        o[j + 2] = __float_as_uint(__uint_as_float(o[j + 2]) * f.z);
                        o[j + 3] = __float_as_uint(__uint_as_float(o[j + 3]) * f.w);
                    }
                    tc::tmem_st32(ta, o);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::named_bar_sync(2, 128);       // alpha is read before the next unit writes it
            }
            tc::fence_proxy_async_smem();
            mbar_arrive(&ctl->p_full[pb]);
            const UnitInfo cur = info;
            const int cslot = slot;
            const uint32_t cpar = par0;
            if (c + 1 < n) {
                if (!(ready & 1u)) {
                    (void)pm_wait(ctl, &ctl->kv_full[nslot], npar);
                    next = ctl->unit[nslot];
                }
                info = next;
            }
            slot2 = slot1; par2 = par1;
            slot1 = slot; par1 = par0;
            slot = nslot; par0 = npar;
            if (!cur.is(kUnitLast)) continue;

            // -------------------------------------------------------------- end of a part
            // The last part is written by all warps, below. Behind any other, every S of
            // the part is done: the next row tile's queries are loaded while the last PV
            // runs, and its products start behind this part's output.
            const bool more = c + 1 < n;
            if (more) load_q(tile + 1, std::integral_constant<int, 2>{});
            bad = !pm_wait(ctl, &ctl->kv_empty[cslot], cpar);   // the part's last PV
            if (owner) ctl->linv[hh] = l != 0.f ? out_scale / l : 0.f;
            if (tc::named_bar_or(2, 128, bad)) { failed = true; break; }
            const int nr = rt.rows(tile);
            const size_t row0 = (size_t)rt.first_row(tile);
            if (cur.part < 0) {
                if (lse && owner && hh < nr)
                    lse[row0 + hh] = l != 0.f ? (m_used + log2f(l)) * 0.6931471805599453f : -INFINITY;
            } else if (owner) {
                part_ml[(size_t)cur.part * kPmRows + hh] = make_float2(m_used, l);
            }
            if (!more) {
                if (tid == 0) {
                    ctl->last_tile = tile;
                    ctl->last_part = cur.part;
                }
                break;
            }
            release_q(tile + 1);
            tc::fence_after_sync();
#pragma unroll 1
            for (int blk = 0; blk < 8; ++blk)
                pm_write_rows(ctl, tl, wq, blk, nr, row0, cur.part, sP + wq * 2048, out, part);
            tc::fence_before_sync();
            tc::named_bar_sync(2, 128);       // linv is read before the next part writes it
            ++tile;
            m_used = -INFINITY;
            l = 0.f;
        }
        if (failed && tid == 0) ctl->last_tile = -1;
        tc::cp_async_wait_all();
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // The last part out of tensor memory: warp w reads the lane quarter w % 4, three
    // warps a quarter sharing its eight pieces.
    const int tile = n > 0 ? ctl->last_tile : -1;
    if (tile >= 0 && warp < 12) {
#pragma unroll 1
        for (int blk = warp >> 2; blk < 8; blk += 3)
            pm_write_rows(ctl, tmem + ((uint32_t)(32 * (warp & 3)) << 16), warp & 3, blk, rt.rows(tile),
                          (size_t)rt.first_row(tile), ctl->last_part, sKV + warp * 2048, out, part);
    }
    // Every MMA of this CTA has completed, and every read, before tensor memory is released.
    if (warp == kPmIssuer) (void)mbar_wait(&ctl->fin, 0);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kPmIssuer) tc::tmem_dealloc(tmem, 512);
}

// Row tiles that were split: entry blockIdx.x, rows_per_block rows a block. A warp
// takes a quarter of the channels of a row (four a lane), eight parts in flight at
// once, and of up to four parts those of two rows; the block's two halves take
// alternate rows. With blocks for each quarter (gridDim.z 4: at most eight row
// tiles, so many parts) the warps of a row, four or eight, share its parts, and the
// first of them merges their sums. The order of the sums depends on the parts alone. Blocks cost
// about 1 ns each even where nothing was split, so there are about a thousand.
constexpr int kMergeWarps = 8;

// Running sums of a row's parts in this lane's four channels.
struct MergeRow {
    float M = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);

    template <int kN>
    DSA_DEVINL void add(const float2 (&ml)[kN], const float4 (&v)[kN]) {
        float Mn = M;
#pragma unroll
        for (int k = 0; k < kN; ++k) Mn = fmaxf(Mn, ml[k].x);
        if (l != 0.f) {
            const float keep = ex2(M - Mn);
            l *= keep; o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
        }
        M = Mn;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if (ml[k].y == 0.f) continue;             // a part without tokens: its row holds nothing
            const float wt = ex2(ml[k].x - M);
            l = fmaf(ml[k].y, wt, l);
            o.x = fmaf(v[k].x, wt, o.x);
            o.y = fmaf(v[k].y, wt, o.y);
            o.z = fmaf(v[k].z, wt, o.z);
            o.w = fmaf(v[k].w, wt, o.w);
        }
    }
    DSA_DEVINL void write(size_t row, int c4, float out_scale, __nv_bfloat16 *out, float *lse) const {
        const bool any = l != 0.f;
        const float inv = any ? out_scale / l : 0.f;
        *reinterpret_cast<uint2 *>(out + row * kL + 4 * c4) =
            any ? make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv))
                : make_uint2(0u, 0u);
        if (lse && c4 == 0) lse[row] = any ? (M + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
};

__global__ void __launch_bounds__(kMergeWarps * 32, 3)
prefix_mla_merge_kernel(const float *__restrict__ part, const float2 *__restrict__ part_ml,
                        const MergeEntry *__restrict__ merge, int Q, int Hm, int rows_per_block,
                        float out_scale, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
    __shared__ float4 so[kMergeWarps][32];
    __shared__ float2 sml[kMergeWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const MergeEntry e = merge[blockIdx.x];
    const RowTiles rt(Q, Hm);
    if (e.tile < 0 || e.tile >= rt.count || e.parts <= 1) return;
    if (e.first_cta < 0 || e.parts > kPmGrid || e.first_cta + e.parts > kPmGrid) return;
    const size_t row0 = (size_t)rt.first_row(e.tile);
    const int rb = blockIdx.y * rows_per_block, r1 = min(rt.rows(e.tile), rb + rows_per_block);
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * e.first_cta + 1 : 2 * (e.first_cta + i)); };
    // parts i0, i0 + step, ... of row r
    auto load = [&](int i0, int step, int r, int c4, auto &ml, auto &v) {
#pragma unroll
        for (int k = 0; k < (int)(sizeof(ml) / sizeof(ml[0])); ++k) {
            const int i = i0 + k * step;
            const bool in = i < e.parts && r < r1;
            ml[k] = in ? part_ml[slot(i) * kPmRows + r] : make_float2(-INFINITY, 0.f);
            v[k] = in ? reinterpret_cast<const float4 *>(part + (slot(i) * kPmRows + r) * kL)[c4]
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    if (gridDim.z == 1) {
        const int c4 = (warp & 3) * 32 + lane, half = warp >> 2;
        if (e.parts <= 4) {
            for (int r = rb + half; r < r1; r += 4) {
                float2 ml[2][4];
                float4 v[2][4];
                load(0, 1, r, c4, ml[0], v[0]);
                load(0, 1, r + 2, c4, ml[1], v[1]);
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    if (r + 2 * a >= r1) break;
                    MergeRow row;
                    row.add(ml[a], v[a]);
                    row.write(row0 + r + 2 * a, c4, out_scale, out, lse);
                }
            }
            return;
        }
        for (int r = rb + half; r < r1; r += 2) {
            MergeRow row;
            for (int i0 = 0; i0 < e.parts; i0 += 8) {
                float2 ml[8];
                float4 v[8];
                load(i0, 1, r, c4, ml, v);
                row.add(ml, v);
            }
            row.write(row0 + r, c4, out_scale, out, lse);
        }
        return;
    }
    const int c4 = blockIdx.z * 32 + lane;               // its four channels
    const int share = rows_per_block == 1 ? kMergeWarps : kMergeWarps / 2, mine = warp & (share - 1);
    const int side = rows_per_block == 1 ? 0 : warp >> 2;
    for (int r0 = rb; r0 < r1; r0 += rows_per_block) {
        const int r = r0 + side;
        MergeRow row;
        for (int i0 = mine; i0 < e.parts; i0 += 8 * share) {
            float2 ml[8];
            float4 v[8];
            load(i0, share, r, c4, ml, v);
            row.add(ml, v);
        }
        so[warp][lane] = row.o;
        if (lane == 0) sml[warp] = make_float2(row.M, row.l);
        __syncthreads();
        if (mine == 0 && r < r1) {
            float2 ml[kMergeWarps];
            float4 v[kMergeWarps];
#pragma unroll
            for (int k = 0; k < kMergeWarps; ++k) {
                ml[k] = k < share ? sml[(warp + k) & (kMergeWarps - 1)] : make_float2(-INFINITY, 0.f);
                v[k] = so[(warp + k) & (kMergeWarps - 1)][lane];
            }
            MergeRow all;
            all.add(ml, v);
            all.write(row0 + r, c4, out_scale, out, lse);
        }
        __syncthreads();
    }
}

// Workspace: partial O rows fp32 [2 x grid][64][512], (m, l) [2 x grid][64],
// merge entries [grid]. It does not grow with the batch.
constexpr size_t kPmPartBytes = (size_t)2 * kPmGrid * kPmRows * kL * sizeof(float);
constexpr size_t kPmMlBytes = (size_t)2 * kPmGrid * kPmRows * sizeof(float2);
inline size_t prefix_mla_workspace_bytes(int Q, int Hm) {
    return Q > 0 && Hm > 0 ? kPmPartBytes + kPmMlBytes + kPmGrid * sizeof(MergeEntry) : 0;
}

// Whether pm_plan's sums hold whatever the lengths on the device turn out to be: the units of
// 32 row tiles in 32 bits, a CTA's share in an int. A tile walks at most its queries' sequences,
// each of them no longer than its table's pages, and two units more a query for their ends.
inline bool pm_sums_fit(const PrefixGeom &g, const RowTiles &rt) {
    const long long held = std::min((long long)std::max(g.prefix_blocks, g.max_blocks) * g.page, (long long)kMaxTokens);
    const long long tile = rt.qpt * (held / kPmTile + 2);
    return std::min(rt.count, 32) * tile <= (long long)UINT32_MAX && rt.count * tile / kPmGrid < INT32_MAX;
}

template <bool kFp8, int kWidth>
inline int prefix_mla_run(const void *q, const void *kv, const PrefixGeom &g, int Hm,
                          float scale_log2, float out_scale, void *out, float *lse, void *ws,
                          cudaStream_t stream) {
    CUtensorMap map = {};
    int box_rows = 0;
    if (!kFp8 && g.page % 16 == 0 && g.kv_rows >= kPmTile) {
        box_rows = g.page % 32 == 0 ? 32 : 16;
        // whole pages of 32 rows: a unit is one box of all its 64-channel atoms
        if (!make_map_bf16_atoms(&map, kv, (uint64_t)g.kv_rows, kWidth / 64, box_rows,
                                 box_rows == kPmTile ? kWidth / 64 : 1))
            return DSA_ERR_CUDA;
    }
    if (!ensure_smem_attr(reinterpret_cast<const void *>(prefix_mla_kernel<kFp8, kWidth>),
                          PmSmem<kFp8, kWidth>::kBytes))
        return DSA_ERR_CUDA;
    auto *part = reinterpret_cast<float *>(ws);
    auto *ml = reinterpret_cast<float2 *>(reinterpret_cast<uint8_t *>(ws) + kPmPartBytes);
    auto *merge = reinterpret_cast<MergeEntry *>(reinterpret_cast<uint8_t *>(ws) + kPmPartBytes + kPmMlBytes);
    auto *ob = reinterpret_cast<__nv_bfloat16 *>(out);
    if (launch_pdl(prefix_mla_kernel<kFp8, kWidth>, dim3(kPmGrid), dim3(pm_threads(kFp8)),
                   PmSmem<kFp8, kWidth>::kBytes, stream, map, box_rows,
                   reinterpret_cast<const __nv_bfloat16 *>(q), kv, g, Hm, scale_log2, out_scale, part,
                   ml, merge, ob, lse) != cudaSuccess)
        return DSA_ERR_CUDA;
    const int st = launch_status();
    if (st != DSA_OK) return st;
    // Up to as many row tiles as CTAs: an entry a tile. More are split at most where a
    // CTA's range ends: an entry a CTA.
    const RowTiles rt(g.Q, Hm);
    const int entries = std::min(rt.count, kPmGrid);
    const bool quarters = rt.count <= 8;
    const int rpb = quarters ? (rt.count <= 2 ? 1 : 2) : std::max(2, 2 * ceil_div((long long)entries * kPmRows, 2 * 1024));
    if (launch_pdl(prefix_mla_merge_kernel, dim3(entries, ceil_div(std::min(kPmRows, rt.total_rows), rpb), quarters ? kL / 128 : 1),
                   dim3(kMergeWarps * 32), 0, stream, part, ml, merge, g.Q, Hm, rpb, out_scale, ob,
                   lse) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}

template <bool kFp8>
inline int prefix_mla_launch(const void *q, const void *kv, float kv_scale, int64_t kv_rows,
                             PrefixGeom g, int Hm, int kv_lora, int rope, float sm_scale, void *out,
                             float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
    if (g.Q < 0 || g.B < 0 || Hm <= 0 || kv_lora <= 0 || rope < 0 || kv_rows < 0 || g.page <= 0 ||
        g.max_blocks < 0 || g.prefix_blocks < 0)
        return DSA_ERR_INVALID_ARG;
    if (!(sm_scale == sm_scale) || sm_scale == INFINITY || sm_scale == -INFINITY)
        return DSA_ERR_INVALID_ARG;
    if (kFp8 && !(kv_scale > 0.f && kv_scale < INFINITY)) return DSA_ERR_INVALID_ARG;
    const float scale_log2 = (kFp8 ? sm_scale * kv_scale : sm_scale) * 1.4426950408889634f;
    if (!(fabsf(scale_log2) < INFINITY)) return DSA_ERR_INVALID_ARG;
    if (kv_lora != DSA_KV_LORA || (rope != 0 && rope != kRopeDim) || Hm % 16 != 0 ||
        Hm > DSA_MAX_MLA_HEADS)
        return DSA_ERR_UNSUPPORTED;
    if (kv_rows > (int64_t)INT32_MAX || g.Q > 65535 || !pm_sums_fit(g, RowTiles(g.Q, Hm)))
        return DSA_ERR_UNSUPPORTED;
    if (g.Q == 0) return DSA_OK;
    if (!q || !g.q_req || !g.q_pos || !out || (kv_rows > 0 && !kv) || (g.B > 0 && !g.seq_len) ||
        (g.B > 0 && g.max_blocks > 0 && !g.block_table) ||
        (g.prefix_blocks > 0 && (!g.prefix_table || !g.prefix_len)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(g.prefix_table, 4) ||
        !aligned(g.prefix_len, 4) || !aligned(g.block_table, 4) || !aligned(g.seq_len, 4) ||
        !aligned(g.q_req, 4) || !aligned(g.q_pos, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(ws, 16))
        return DSA_ERR_ALIGNMENT;
    if (!ws || ws_bytes < prefix_mla_workspace_bytes(g.Q, Hm)) return DSA_ERR_WORKSPACE;
    g.kv_rows = (int)kv_rows;
    g.page_shift = -1;
    if ((g.page & (g.page - 1)) == 0)
        for (g.page_shift = 0; (1 << g.page_shift) < g.page;) ++g.page_shift;
    const float out_scale = kFp8 ? kv_scale : 1.0f;
    return rope ? prefix_mla_run<kFp8, DSA_KV_LORA + kRopeDim>(q, kv, g, Hm, scale_log2, out_scale,
                                                               out, lse, ws, stream)
                : prefix_mla_run<kFp8, DSA_KV_LORA>(q, kv, g, Hm, scale_log2, out_scale, out, lse, ws,
                                                    stream);
}

}  // namespace dsa
