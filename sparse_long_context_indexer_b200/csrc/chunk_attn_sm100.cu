// chunk_attn_sm100.cu -- attention of a chunk of new tokens over a paged latent cache (MQA mode):
//   out[t,h,:] = sum_{s < n_t} softmax_s(scale * q[t,h,:] . c[s,:]) c[s,0:512],  lse = ln sum exp
// with c[s] the 576-value latent row of position s of row t's sequence, found through the block
// table, and n_t = q_len[t] (which carries the causal mask).
//
// What bounds it.  A row and position cost 2 * 128 * (576 + 512) = 278,528 operations against
// 1,152 bytes, shared by all rows of a sequence: chunks are bound by the tensor cores, and a single
// token a sequence sits where both limits meet (242 operations a byte against 252 at the measured
// rates).  M = 64 MMAs of one SM run at half the tensor rate, and a full 128 x 512 fp32 output fills
// an SM's tensor memory, leaving none for the scores.  So a row is one CTA pair's (cta_group::2,
// M = 128): each CTA holds 64 heads, whose 64 x 512 output takes 256 TMEM columns, and the pair runs
// at the full rate.
//
// A tile is 128 positions.  CTA r of the pair
//   * loads rows 64 r .. 64 r + 63 of the tile (the N = 128 half it supplies to S = Q K^T), nine
//     swizzled tiles of 64 rows x 64 values; the ninth (the rotated values) has a slot of its own,
//     the others fill pairs of tiles in a ring of eleven 16 KB slots;
//   * supplies value columns 256 r .. 256 r + 255 of all 128 rows to O += P V.  For its own rows
//     those are already in the ring (pairs 2 r and 2 r + 1); once S is done it overwrites the other
//     two pairs with the other CTA's rows' same columns, so that each MMA finds both CTAs' operand
//     at one offset.  This reads 104 KB a tile instead of 136 KB and needs no second value buffer.
// TMEM columns: O [0, 256) (lanes 0..63 value columns 0..255, lanes 64..127 value columns 256..511),
// S [256, 320) (lanes 0..63 positions 0..63, lanes 64..127 positions 64..127), Q values 0..383
// [320, 512), twice (lanes 0..63 and 64..127); Q values 384..575 stay in shared memory.
//
// Roles of a CTA:
//   warps 0..3  softmax: thread = (head, half of the positions); the two threads of a head exchange
//               the tile's maximum through shared memory.  exp2 domain, O rescaled only when the
//               running maximum grows by more than 8 (a factor 256).  P goes to shared memory in the values' 16-bit type, since
//               the tensor core takes both operands in one: in bf16 off by up to 2^-8 of itself, at random, so that out's
//               error is up to a quarter above that of its own rounding.  Sums are fp32, of P as it was before.
//   warps 4..7  outputs, those of empty rows too
//   warp 8      by TMA, this CTA's rows of the tiles, and before a row's tiles its query block: values 0..383
//               through three ring entries, from where the tensor core copies them into TMEM, twice
//   warp 9      (leader) MMA issue: Q K^T of tile i + 1 goes out before P V of tile i
//   warp 10     the other CTA's rows' value columns, by TMA
// FP8 entries (656 bytes) have no tiles that TMA could fetch: eight warps read the codes and write
// fp16 tiles themselves, in the same slots and order (1.5 x 512 values a row).
// A tile that ends inside (or names a block outside the pool) may bring anything: masked scores
// are replaced, and the softmax warps zero the masked rows of V before P V, since 0 * NaN is NaN.
//
// Work split.  All rows' tiles in a line (with some units for a row itself), one equal piece per pair, so
// that one long row spreads over every SM and a thousand short ones balance alike.  A row that crosses
// pieces leaves normalised fp32 partials (two slots a pair) that chunk_combine_kernel merges in the order
// of the positions: results do not depend on timing.
//
// Measured (fresh inputs each time): 512 rows after 8,192 positions 1.0 ms (1.2 PFLOP/s; a library product of
// matrices sustains 1.4 under the same power cap), 2,048 rows after 30,001 13.9 ms (1.27 PFLOP/s), 32 single
// tokens of 16 to 32 K positions 0.26 ms (3.6 TB/s); over FP8 entries 300 rows after 12,345 1.2 ms (0.85 PFLOP/s),
// after 1,700 0.32 ms (0.48), 24 single tokens of 8 to 16 K 0.14 ms; one row of 701 positions 16 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kHalf = 64;                        // positions a CTA loads per tile
constexpr int kHeads = 64;                       // heads per CTA
constexpr int kSub = 64 * 128;                   // one tile of 64 rows x 64 bf16
constexpr int kPair = 2 * kSub;
constexpr int kRing = 11;                        // slots of two tiles
constexpr int kOffRing = 0;
constexpr int kOffRope = kOffRing + kRing * kPair;
constexpr int kOffQ = kOffRope + kSub;           // Q values 384..575: three tiles of 64 heads
constexpr int kOffP = kOffQ + 3 * kSub;          // P: two tiles of 64 heads x 64 positions
constexpr int kOffMax = kOffP + 2 * kSub;        // [2 tiles][2 halves][64 heads]
constexpr int kOffStat = kOffMax + 4 * kHeads * 4;  // [2 pieces][sum of each half, maximum][64 heads]
constexpr int kOffBar = kOffStat + 6 * kHeads * 4;
// barriers, in 8-byte units from kOffBar
constexpr int kBarPairFull = 0;                  // [kRing] leader
constexpr int kBarPairEmpty = kBarPairFull + kRing;
constexpr int kBarRopeFull = kBarPairEmpty + kRing;  // leader
constexpr int kBarRopeEmpty = kBarRopeFull + 1;
constexpr int kBarV = kBarRopeEmpty + 1;         // [2] leader
constexpr int kBarVTail = kBarV + 2;             // [2]
constexpr int kBarS = kBarVTail + 2;             // [2]
constexpr int kBarSFree = kBarS + 2;             // leader
constexpr int kBarP = kBarSFree + 1;             // leader
constexpr int kBarO = kBarP + 1;
constexpr int kBarOFree = kBarO + 1;             // leader
constexpr int kBarQ = kBarOFree + 1;             // leader
constexpr int kBarQFree = kBarQ + 1;
// [2] by the parity of the piece: the output warps may still be on their way to a piece (past many empty rows, say)
// when the softmax warps have ended the next one, and a barrier two phases ahead looks like one that has not come.
// The second next waits for the outputs of this one (kBarOFree).
constexpr int kBarStat = kBarQFree + 1;
constexpr int kNumBars = kBarStat + 2;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;

// warps over a bf16 cache: 0..3 softmax, 4..7 outputs, 8 this CTA's rows and the queries, 9 MMA issue, 10 the
// other's rows; over FP8 entries: 0..3 softmax, queries and outputs, 4..11 both kinds of rows, 12 MMA issue
constexpr int kThreadsBf16 = 352, kThreadsFp8 = 512;
// register split over FP8 entries (512 threads start with 128 each): the softmax warpgroup takes what the
// issuing warpgroup gives, 176 + 128 + 128 + 80 = 4 * 128
constexpr int kRegsSoftmax = 176, kRegsIssue = 80;
static_assert(kRegsSoftmax + 2 * 128 + kRegsIssue <= 4 * 128, "the launch's registers");
constexpr int kMaxWarps = kThreadsFp8 / 32;
static_assert(2 * kMaxWarps * 8 <= 4 * kHeads * 4 && kOffMax % 8 == 0, "the plan's sums in the maxima's place");
constexpr int kDequantWarps = 8;
struct Shared {
    int tmem_base;
    int abort_flag;
    int row0, skip;                              // first row of this pair's piece, units of it before the piece
    int count;                                   // units of the piece
    int pieces;                                  // pairs that have work
    int base;                                    // first pair of those that share this pair's kind of rows
    int two;                                     // that kind: scores of two terms (kMixed)
    long long lo, total;                         // (of the kind's line of units)
};
constexpr int kSmemBytes = kOffMisc + (int)sizeof(Shared);  // from a 1 KB boundary (the swizzle's period)
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
static_assert(kOffMisc % 8 == 0, "alignment of the shared scalars");

constexpr uint32_t kColS = 256, kColQ = 320;
constexpr int kQEntries = 3;                     // ring entries of a piece's query tiles (bf16 cache)
constexpr int kQTmem = 6;                        // 64-value tiles of Q kept in TMEM
constexpr float kRescale = 8.0f;                 // log2 units
// The FP8 cache is worked on in fp16 (operand format 0): its values, e4m3 code times fp32 scale, lose
// 2^-10 there (two roundings) against 2^-8 in bf16, and P 2^-11.  P is kept 2^7 times larger (at most 2^15
// with the deferred rescaling), which moves fp16's smallest step to 2^-31 of the row's maximum.
constexpr float kFp16Bias = 7.0f;
// A score over fp16 values is off by up to 2^-10 of its products' size: by 4e-4 for random values (q and c of size 1, scale
// 1 / sqrt(192)), by 1e-4 of itself where the products add up (the rounding of a group's scale is the same for its 128
// values: 4e-3 at a score of 40).  Where a row's weights spread over many positions that averages out of lse (4e-5 over 4,000
// random ones, 2.5e-5 over 12,000); where they sit on one it does not, and weights of out are off by as much.
// A row of up to kTwoTerms positions therefore has its values as a sum of two fp16 terms in Q K^T (off by 2^-20; lse
// of random values by 2e-6): a tile's low terms pass through four ring entries of their own before the tile itself,
// 32 MMAs more (300 rows after 1,700 positions 322 instead of 221 us).  Longer rows, which a second term would cost
// half as much again (300 after 12,345 1,775 instead of 1,085 us, 24 single tokens of 8 to 16 K 203 instead of 139), keep
// one.  P V takes the first term alone: out is bf16.
constexpr int kTwoTerms = 4096;
// The choice goes by the row's own length, whatever else is in the call or in the table.  A CTA pair has rows of one kind
// only, and the kernel for tables of more than kTwoTerms positions (kMixed) holds the converting and the issuing warps'
// loops in both forms: 144 us for the 24 tokens (139 in a kernel of one form), 1,090 for the 300 rows (1,085).  A
// choice from row to row within a pair costs the long rows 15 to 25 %, two launches one after the other 10 us.  Pairs
// are shared out as the kinds' work, a tile with two terms counting kTwoCost / kOneCost of one without.
constexpr int kTwoCost = 13, kOneCost = 8;

constexpr uint32_t idesc_qk(bool fp8) { return make_idesc(128, 128, fp8 ? 0 : 1, fp8 ? 0 : 1, 0, 0); }
constexpr uint32_t idesc_pv(bool fp8) { return make_idesc(128, 256, fp8 ? 0 : 1, fp8 ? 0 : 1, 0 /*A K-major*/, 1 /*B MN-major*/); }

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// two bf16 values in fp16
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t u) {
    return pack_f16x2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// 4 x 4 transpose of two-word units between the four lanes of a quad: lane j's unit i becomes lane i's unit j.
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4][2], int j) {
#pragma unroll
    for (int step = 1; step <= 2; step <<= 1) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (m & step) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, (j & step) ? x[m][e] : x[m + step][e], step);
                if (j & step)
                    x[m][e] = got;
                else
                    x[m + step][e] = got;
            }
        }
    }
}

// Tiles of row t; 0 for an empty row and for one whose length or sequence is out of range.
__device__ __forceinline__ bool row_ok(const ChunkArgs& a, int n, int b) {
    return n >= 0 && n <= a.T_max && b >= 0 && b < a.B;
}
__device__ __forceinline__ int tiles_of(const ChunkArgs& a, int n, int b) {
    return row_ok(a, n, b) ? (n + kChunkTile - 1) / kChunkTile : 0;
}

// A row's scores over FP8 entries take two terms: a matter of its own length, whatever else is in the call or the table.
__device__ __forceinline__ bool two_terms(int n) { return n <= kTwoTerms; }

// The work's measure.  Beside its tiles a row costs its query block, the first tile's way through the
// pipeline and its output, so that 512 rows of up to four tiles would leave the pairs with short rows working
// twice as long as the others: a row counts as kRowUnits more.  Measured over a bf16 cache with three, four, five and six (us, in a
// graph): 64 rows after 200 tokens 25.0, 25.0, 20.9, 21.3; 128 after 200 33.2, 32.8, 31.2, 31.6; 64 single tokens
// of 1,001 positions 41.4, 41.4, 39.7, 39.3; 512 rows of one prompt 76.2, 77.0, 77.6, 78.1; 300 rows after 2,000 156.1, 155.8, 155.4, 154.5.
constexpr int kRowUnits = 5;
__device__ __forceinline__ int units_of(int tiles) { return tiles == 0 ? 0 : tiles + kRowUnits; }

// Units that a piece of long rows has at least: a row of many one-tile pieces costs more to merge than its tiles
// save (one row of 8,001 positions 25.1 us in pieces of one unit, 21.5 of two, 21.1 of three, 23 of four; of 12,001
// 26.6, 24.1, 21.8, 23.4; over FP8 entries, whose tiles take longer, in a graph, of 8,001 31.6, 27.0, 31.1, 31.1, of
// 12,001 33.2, 29.5, 29.1, 33.2).  Rows of less than 16 units on average are cut as finely as they come (8 rows of 501
// positions 16.7 us in pieces of one unit, 19.4 of three).
template <bool kFp8>
__device__ __forceinline__ int min_piece() {
    return kFp8 ? 2 : 3;
}

// The pair's piece of the line of units, row by row: tiles [i0, i1) of `row` (a row's own units come before
// its tiles).  The row after the current one is read ahead of its use.
template <bool kFp8, bool kMixed>
struct Pieces {
    const ChunkArgs& a;
    int row, n, b, nt, i0, i1, left, skip;
    int n_next, b_next;
    bool two;  // its rows' scores take two terms
    __device__ __forceinline__ Pieces(const ChunkArgs& args, const Shared* sh) : a(args) {
        row = sh->row0 - 1;
        left = sh->count;
        skip = sh->skip;
        two = kMixed ? sh->two != 0 : kFp8;
        i0 = i1 = 0;
        n = b = nt = 0;
        n_next = b_next = 0;
        if (left > 0) {
            n_next = __ldg(a.q_len + sh->row0);
            b_next = __ldg(a.q_seq + sh->row0);
        }
    }
    __device__ __forceinline__ bool next() {
        do {
            if (left <= 0) return false;
            do {
                if (++row >= a.Nq) return false;  // only if the lengths changed under the kernel
                n = n_next;
                b = b_next;
                nt = tiles_of(a, n, b);
                if (kMixed && two_terms(n) != two) nt = 0;  // (another pair's)
                if (row + 1 < a.Nq) {
                    n_next = __ldg(a.q_len + row + 1);
                    b_next = __ldg(a.q_seq + row + 1);
                }
            } while (nt == 0);
            const int own = units_of(nt) - nt, take = min(nt + own - skip, left);
            left -= take;
            i0 = max(0, skip - own);
            i1 = max(0, skip + take - own);
            skip = 0;
        } while (i1 <= i0);  // (a piece that ends within a row's own units has none of its tiles)
        return true;
    }
};

// Positions [64 h, 64 h + 64) of tile i of a row: how many take part, and their first pool row
// (0 when none does: a load then brings rows that are masked).
struct HalfTile {
    int lim, row;
    bool bad;
};
__device__ __forceinline__ int half_block(const ChunkArgs& a, const int32_t* tab, int n, int i, int h) {
    const int s0 = i * kChunkTile + h * kHalf;
    return s0 < n ? __ldg(tab + (s0 >> a.block_shift)) : -1;
}
__device__ __forceinline__ HalfTile half_tile(const ChunkArgs& a, int pb, int n, int i, int h) {
    const int s0 = i * kChunkTile + h * kHalf;
    HalfTile t;
    const bool in = s0 < n, ok = in && pb >= 0 && pb < a.num_blocks;
    t.bad = in && !ok;
    t.lim = ok ? min(kHalf, n - s0) : 0;
    t.row = ok ? (pb << a.block_shift) + (s0 & ((1 << a.block_shift) - 1)) : 0;
    return t;
}

// A warp waits until every lane's barrier (0: none) has completed its phase; false when the budget ran out or
// another role gave up.
__device__ __forceinline__ bool wait_lanes(uint32_t b, int parity, int lane, volatile int* abort_flag, int* status) {
    const uint64_t t0 = globaltimer_ns();
    uint32_t spins = 0;
    while (true) {
        if (__all_sync(0xffffffffu, b == 0 || mbar_test(b, parity))) return true;
        if ((++spins & 255u) == 0) {
            bool stop = *abort_flag != 0;
            if (!stop && globaltimer_ns() - t0 > kWaitBudgetNs) {
                if (lane == 0) {
                    record_status(status, DSA_STATUS_TIMEOUT);
                    *abort_flag = 1;
                }
                stop = true;
            }
            if (__any_sync(0xffffffffu, stop)) return false;
        }
    }
}

// All roles of a CTA over its pair's piece of the rows.
template <bool kFp8, bool kMixed>
__device__ __forceinline__ void chunk_roles(const ChunkArgs& a, const CUtensorMap& map_pair, const CUtensorMap& map_rope,
                                            const CUtensorMap& map_q, const CUtensorMap& map_q3, const uint32_t sb, Shared* sh,
                                            const bool empty_rows) {
    constexpr uint32_t kIdescQK = idesc_qk(kFp8), kIdescPV = idesc_pv(kFp8);
    constexpr float kBias = kFp8 ? kFp16Bias : 0.f;
    constexpr int kMmaWarp = kFp8 ? 12 : 9;
    volatile int* abort_flag = &sh->abort_flag;
    auto bar = [&](int i) { return sb + kOffBar + 8u * i; };
    auto pair_addr = [&](int n) { return sb + kOffRing + (uint32_t)(n % kRing) * kPair; };
    // ring entry of pair 0 of the pair's tile g in its piece `seg`: over a bf16 cache three entries with query
    // tiles come before a piece's tiles, with two terms a tile's low terms before the tile
    auto entry_of = [](int g, int seg, bool two = false) { return two ? 8 * g + 4 : 4 * g + (kFp8 ? 0 : kQEntries * (seg + 1)); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_ctarank();
    const int cluster = blockIdx.x >> 1;
    const bool leader = rank == 0;
    auto lead = [&](int i) { return mapa_shared(bar(i), 0); };  // the leader's barrier
    const uint32_t tmem = (uint32_t)sh->tmem_base;
    Pieces<kFp8, kMixed> pc(a, sh);

    // ---- outputs out: four warps (4..7 over a bf16 cache; over FP8 entries the softmax warps, queries in too)
    bool ok = true;  // a wait of these roles ran out: the loops go on without touching memory, so that
                     // every warp still meets the others at the named barriers
    const int io_warp = warp & 3, p = tid & 127, r = (io_warp & 1) * 32 + lane;  // head of this lane
    const uint32_t lanes = tmem + ((uint32_t)(io_warp * 32) << 16);
    int started = -1, started_row = 0, started_rest = 0;  // slot of the piece whose row goes on in the next pair, and
                                                          // the row's tiles that are left there
    // Over FP8 entries the query block becomes fp16 on its way: three sets of three 64-value tiles, read coalesced;
    // once the piece before has its last Q K^T, sets 0 and 1 pass through the shared tiles into TMEM, a head a
    // lane, and set 2 stays in the shared tiles.  (Over a bf16 cache TMA brings it and the tensor core copies.)
    struct Piece {
        int row, i0, rest, end;  // first tile, the row's tiles after the piece, the pair's tiles up to its end
    };
    // granule e of a set: head e / 24, 16 bytes e % 24 of its 384
    auto load_q = [&](uint4 (&d)[12], int row, int set) {
        const uint4* src = reinterpret_cast<const uint4*>(
            reinterpret_cast<const __nv_bfloat16*>(a.q) + ((int64_t)row * kMlaHeads + rank * kHeads) * kDK);
#pragma unroll
        for (int k = 0; k < 12; ++k) {
            const int e = p + 128 * k, hd = e / 24, gr = e - hd * 24;
            d[k] = __ldg(src + hd * (kDK / 8) + set * 24 + gr);
        }
    };
    // q0 holds set 0
    auto stage_q = [&](uint4 (&q0)[12], int row, int seg) {
        auto to_shared = [&](const uint4 (&d)[12]) {
#pragma unroll
            for (int k = 0; k < 12; ++k) {
                const int e = p + 128 * k, hd = e / 24, gr = e - hd * 24;
                const uint32_t dst = sb + kOffQ + (gr >> 3) * kSub + hd * 128 + (((gr & 7) ^ (hd & 7)) << 4);
                st_shared_v4(dst, bf16x2_to_f16x2(d[k].x), bf16x2_to_f16x2(d[k].y), bf16x2_to_f16x2(d[k].z),
                             bf16x2_to_f16x2(d[k].w));
            }
        };
        auto to_tmem = [&](int set) {
#pragma unroll 1
            for (int c = 0; c < 3; ++c) {
                uint32_t w[32];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[4 * k]), "=r"(w[4 * k + 1]), "=r"(w[4 * k + 2]), "=r"(w[4 * k + 3])
                                 : "r"(sb + kOffQ + c * kSub + r * 128 + ((k ^ (r & 7)) << 4))
                                 : "memory");
                tmem_st32(lanes + kColQ + 32 * (3 * set + c), w);
            }
        };
        const uint32_t q_full = lead(kBarQ);
        if (seg > 0 && ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarQFree), (seg - 1) & 1, abort_flag, a.status));
            tc_fence_after();
        }
#pragma unroll 1
        for (int set = 0; set < 2; ++set) {
            if (ok) to_shared(q0);
            load_q(q0, row, set + 1);
            named_barrier_sync(3, 128);
            if (ok) to_tmem(set);
            named_barrier_sync(3, 128);
        }
        if (ok) {
            to_shared(q0);
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(q_full);
        }
    };
    // the output of piece `s`: out = O / l, or fp32 for the merge
    auto output = [&](int s, const Piece& pi) {
        const bool whole = pi.i0 == 0 && pi.rest == 0;
        const int row = pi.row;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarStat + (s & 1)), (s >> 1) & 1, abort_flag, a.status));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_spin(bar(kBarO), (pi.end - 1) & 1, abort_flag, a.status));
        if (!ok) return;
        tc_fence_after();
        const int half = io_warp >> 1, head = rank * kHeads + r;
        const uint32_t st = sb + kOffStat + (s & 1) * (3 * kHeads * 4);
        auto sum_of = [&](int rr) { return ld_shared_f32(st + rr * 4) + ld_shared_f32(st + (kHeads + rr) * 4); };
        const float l = sum_of(r), m = ld_shared_f32(st + (2 * kHeads + r) * 4);
        // (a sum of 0: no position; NaN stays NaN)
        const float lse = l == 0.f ? -CUDART_INF_F : (m - kBias + __log2f(l)) * 0.6931471805599453f;
        // a pair's first piece has slot 0; any other is its last: slot 1
        const int slot = 2 * cluster + (s == 0 ? 0 : 1);
        if (half == 0) {
            if (!whole)
                a.part_lse[slot * kMlaHeads + head] = lse;
            else if (a.lse)
                a.lse[(int64_t)row * kMlaHeads + head] = lse;
        }
        if (!whole && pi.i0 == 0) started = slot, started_row = row, started_rest = pi.rest;
        // Blocks of 16 heads x 64 values: a lane gets columns 8 k + 2 j, + 1 (k = 0..7, j = lane % 4) of heads
        // lane / 4 and that + 8; the four lanes of a head exchange until each has 32 contiguous bytes, so that
        // a store instruction covers whole lines (with a lane a head it touches 32 of them, in the way of the other
        // roles' accesses: 512 rows after 8,192 tokens 1,039 instead of 998 us).
        const int j = lane & 3, r4 = (io_warp & 1) * 32 + (lane >> 2);
        __nv_bfloat16* o16 = reinterpret_cast<__nv_bfloat16*>(a.out) + ((int64_t)row * kMlaHeads + rank * kHeads) * kDV + half * 256;
        float* o32 = a.part_o + ((int64_t)slot * kMlaHeads + rank * kHeads) * kDV + half * 256;
#pragma unroll 1
        for (int b = 0; b < 8; ++b) {
            const int c0 = 64 * (b & 3), r0 = r4 + 16 * (b >> 2);
            uint32_t ov[32];
            tmem_ld16x256b_x8(lanes + ((uint32_t)(16 * (b >> 2)) << 16) + c0, ov);
            float inv[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float x = sum_of(r0 + 8 * q);
                inv[q] = x == 0.f ? 0.f : 1.f / x;
            }
            tmem_wait_ld_regs(ov);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t at = (int64_t)(r0 + 8 * q) * kDV + c0;
                if (whole) {
                    uint32_t x[4][2];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        x[k & 3][k >> 2] = pack_bf16x2(__uint_as_float(ov[4 * k + 2 * q]) * inv[q],
                                                       __uint_as_float(ov[4 * k + 2 * q + 1]) * inv[q]);
                    quad_transpose(x, j);
                    uint4* o = reinterpret_cast<uint4*>(o16 + at + 8 * j);
                    o[0] = make_uint4(x[0][0], x[1][0], x[2][0], x[3][0]);
                    o[4] = make_uint4(x[0][1], x[1][1], x[2][1], x[3][1]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t x[4][2];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                x[k][e] = __float_as_uint(__uint_as_float(ov[16 * h + 4 * k + 2 * q + e]) * inv[q]);
                        quad_transpose(x, j);
                        const uint32_t w[8] = {x[0][0], x[0][1], x[1][0], x[1][1], x[2][0], x[2][1], x[3][0], x[3][1]};
                        st_global_v8(o32 + at + 32 * h + 8 * j, w);
                    }
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(kBarOFree));
    };
    auto finish = [&]() {
        if (leader && p == 0) {
            // the row that starts here and goes on: it ends in the pair that has its last tile
            int4 meta = make_int4(-1, 0, 0, 0);
            if (ok && started >= 0) {
                const long long end = sh->lo + sh->count + started_rest;  // one past the row's last unit
                int c = cluster - sh->base + 1;
                while (sh->total * (c + 1) / sh->pieces < end) ++c;
                meta = make_int4(started_row, started, sh->base + c, 0);
            }
            a.meta[cluster] = meta;
        }
        if (empty_rows) {
            for (int t = cluster; t < a.Nq; t += a.clusters) {
                if (tiles_of(a, __ldg(a.q_len + t), __ldg(a.q_seq + t)) != 0) continue;
                const int64_t first = (int64_t)t * kMlaHeads + rank * kHeads;
                uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + first * kDV);
                for (int e = p; e < kHeads * kDV / 8; e += 128) o[e] = make_uint4(0u, 0u, 0u, 0u);
                if (a.lse && p < kHeads) a.lse[first + p] = -CUDART_INF_F;
            }
        }
    };

    if (warp < 4) {
        if constexpr (kFp8) setmaxnreg_inc<kRegsSoftmax>();
        // ------------------------------------------------ softmax
        const int half = warp >> 1;  // of the positions
        // (a zero scale becomes one that leaves every finite score at zero and a masked one at -inf)
        const float scale = a.softmax_scale == 0.f ? 1e-37f : a.softmax_scale * 1.4426950408889634f;
        const uint32_t masked = scale > 0.f ? 0xFF800000u : 0x7F800000u;  // -inf once multiplied
        const uint32_t p_row = sb + kOffP + half * kSub + r * 128;
        const uint32_t s_free = lead(kBarSFree), p_full = lead(kBarP);
        int g = 0, seg = 0;
        int tails[2] = {0, 0};  // by the parity of the tile: two tiles in a row may end inside (bad blocks), and the second
                                // one's rows may land before this warp looks for the first one's
        Piece last{0, 0, 0, 0};
        auto wait = [&](int i, int parity) {
            // (a test in a loop answers sooner than a blocking wait, 512 rows after 8,192 tokens 1,025 -> 1,005 us; beside
            // the dequantising warps its polls cost more than they save: 300 rows after 12,000 1,202 -> 1,217 us)
            if (ok)
                ok = kFp8 ? (bool)__all_sync(0xffffffffu, mbar_wait_spin(bar(i), parity, abort_flag, a.status))
                          : wait_lanes(lane == 0 ? bar(i) : 0u, parity, lane, abort_flag, a.status);
            if (ok) tc_fence_after();
        };
        while (pc.next()) {
            if constexpr (kFp8) {
                uint4 q0[12];
                load_q(q0, pc.row, 0);
                stage_q(q0, pc.row, seg);
                if (seg > 0) output(seg - 1, last);
                last = Piece{pc.row, pc.i0, pc.nt - pc.i1, g + pc.i1 - pc.i0};
            }
            const int32_t* tab = a.block_table + (int64_t)pc.b * a.max_blocks;
            float m = -CUDART_INF_F, l = 0.f;
            int pb0 = half_block(a, tab, pc.n, pc.i0, 0), pb1 = half_block(a, tab, pc.n, pc.i0, 1);
            for (int i = pc.i0; i < pc.i1; ++i, ++g) {
                const HalfTile h0 = half_tile(a, pb0, pc.n, i, 0), h1 = half_tile(a, pb1, pc.n, i, 1);
                if (i + 1 < pc.i1) {
                    pb0 = half_block(a, tab, pc.n, i + 1, 0);
                    pb1 = half_block(a, tab, pc.n, i + 1, 1);
                }
                const int lim = half ? h1.lim : h0.lim;
                uint32_t s0[32], s1[32];
                float mx = -CUDART_INF_F;
                wait(kBarS + (g & 1), (g >> 1) & 1);
                if (ok) {
                    tmem_ld32(lanes + kColS, s0);
                    tmem_ld32(lanes + kColS + 32, s1);
                    tmem_wait_ld_regs(s0);
                    tmem_wait_ld_regs(s1);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(s_free);
                    if (lim < kHalf) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            if (c >= lim) s0[c] = masked;
                            if (c + 32 >= lim) s1[c] = masked;
                        }
                    }
                    // the largest score: of the products for a positive scale, the smallest for a negative one
                    float hi = __uint_as_float(s0[0]);
                    if (scale > 0.f) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) hi = fmaxf(hi, fmaxf(__uint_as_float(s0[c]), __uint_as_float(s1[c])));
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) hi = fminf(hi, fminf(__uint_as_float(s0[c]), __uint_as_float(s1[c])));
                    }
                    mx = hi * scale;
                }
                const uint32_t xm = sb + kOffMax + (g & 1) * (2 * kHeads * 4);
                st_shared_f32(xm + (half * kHeads + r) * 4, mx);
                named_barrier_sync(1 + (warp & 1), 64);
                if (!ok) continue;
                mx = fmaxf(mx, ld_shared_f32(xm + ((half ^ 1) * kHeads + r) * 4));
                const float m_old = m;
                const bool grow = mx > m + kRescale;
                if (grow) m = mx;
                const float sub = m == -CUDART_INF_F ? 0.f : m - kBias;
                uint32_t pk[32];
                const uint64_t scale2 = pack_f32x2(scale, scale), sub2 = pack_f32x2(-sub, -sub);
                uint64_t sum2 = 0;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const uint32_t u = c < 16 ? s0[(2 * c) & 31] : s1[(2 * c) & 31], v = c < 16 ? s0[(2 * c + 1) & 31] : s1[(2 * c + 1) & 31];
                    float p0, p1;
                    unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(u), __uint_as_float(v)), scale2, sub2), p0, p1);
                    p0 = fast_exp2(p0);
                    p1 = fast_exp2(p1);
                    sum2 = add_f32x2(sum2, pack_f32x2(p0, p1));
                    pk[c] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                }
                float sum, sum_odd;
                unpack_f32x2(sum2, sum, sum_odd);
                sum += sum_odd;
                // P's buffer and O are free once P V of the tile before has completed
                if (g > 0) wait(kBarO, (g - 1) & 1);
                if (!ok) continue;
                const bool rescale = grow && m_old != -CUDART_INF_F;
                if (__any_sync(0xffffffffu, rescale)) {
                    const float alpha = rescale ? fast_exp2(m_old - m) : 1.f;
#pragma unroll 1
                    for (int c0 = 0; c0 < 256; c0 += 32) {
                        uint32_t ov[32];
                        tmem_ld32(lanes + c0, ov);
                        tmem_wait_ld_regs(ov);
#pragma unroll
                        for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
                        tmem_st32(lanes + c0, ov);
                    }
                    tmem_wait_st();
                    l *= alpha;
                }
                l += sum;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    st_shared_v4(p_row + ((q ^ (r & 7)) << 4), pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                if (!kFp8 && (h0.lim < kHalf || h1.lim < kHalf)) {
                    // masked rows of V become zeros once both CTAs' rows have landed
                    wait(kBarVTail + (g & 1), tails[g & 1] & 1);
                    if (!ok) continue;
                    ++tails[g & 1];
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        const int lo_row = v ? h1.lim : h0.lim, cells = (kHalf - lo_row) * 32;
                        for (int c = tid; c < cells; c += 128) {
                            const int sub_tile = (c >> 3) & 3;
                            st_shared_v4(pair_addr(entry_of(g, seg) + 2 * v + (sub_tile >> 1)) + (sub_tile & 1) * kSub +
                                             (lo_row + (c >> 5)) * 128 + (c & 7) * 16,
                                         0u, 0u, 0u, 0u);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(p_full);
            }
            // ---- the row's (or piece's) sums and maximum go to the output warps
            const uint32_t st = sb + kOffStat + (seg & 1) * (3 * kHeads * 4);
            st_shared_f32(st + (half * kHeads + r) * 4, l);
            if (half == 0) st_shared_f32(st + (2 * kHeads + r) * 4, m);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarStat + (seg & 1)));
            ++seg;
        }
        if constexpr (kFp8) {
            if (seg > 0) output(seg - 1, last);
            finish();
        }
    } else if (!kFp8 && warp < 8) {
        // ------------------------------------------------ outputs
        int seg = 0, end = 0;
        while (pc.next()) {
            end += pc.i1 - pc.i0;
            output(seg, Piece{pc.row, pc.i0, pc.nt - pc.i1, end});
            ++seg;
        }
        finish();
    } else if (!kFp8 && warp == 8) {
        // ------------------------------------------------ this CTA's rows of every tile
        if (lane == 0) {
            int g = 0, seg = 0;
            bool ok = true;
            // a ring entry: its slot's barrier, once the slot is free
            auto claim = [&](int n) {
                const int slot = n % kRing, use = n / kRing;
                if (use > 0) ok = mbar_wait_spin(bar(kBarPairEmpty + slot), (use - 1) & 1, abort_flag, a.status);
                if (ok && leader) mbar_arrive_expect_tx(bar(kBarPairFull + slot), 2 * kPair);
                return lead(kBarPairFull + slot);
            };
            while (ok && pc.next()) {
                const int32_t* tab = a.block_table + (int64_t)pc.b * a.max_blocks;
                const int q_row = pc.row * kMlaHeads + rank * kHeads;
                int pb = half_block(a, tab, pc.n, pc.i0, rank);
                for (int j = 0; j < kQEntries && ok; ++j) {
                    const int n = entry_of(g, seg) - kQEntries + j;
                    const uint32_t full = claim(n);
                    if (ok) tma_load_3d_pair(pair_addr(n), &map_q, 0, q_row, 2 * j, full);
                }
                for (int i = pc.i0; i < pc.i1 && ok; ++i, ++g) {
                    const HalfTile t = half_tile(a, pb, pc.n, i, rank);
                    if (i + 1 < pc.i1) pb = half_block(a, tab, pc.n, i + 1, rank);
                    if (t.bad) record_status(a.status, DSA_STATUS_INDEX_OOB);
                    for (int j = 0; j < 4 && ok; ++j) {
                        const int n = entry_of(g, seg) + j;
                        const uint32_t full = claim(n);
                        if (ok) tma_load_3d_pair(pair_addr(n), &map_pair, 0, t.row, 2 * j, full);
                    }
                    // the rotated values' slot and query values 384..575 are free once the tile (the piece)
                    // before has its Q K^T
                    if (ok && i == pc.i0) {
                        if (seg > 0) ok = mbar_wait_spin(bar(kBarQFree), (seg - 1) & 1, abort_flag, a.status);
                        if (!ok) break;
                        if (leader) mbar_arrive_expect_tx(bar(kBarQ), 2 * 3 * kSub);
                        tma_load_3d_pair(sb + kOffQ, &map_q3, 0, q_row, kQTmem, lead(kBarQ));
                    }
                    if (ok && g > 0) ok = mbar_wait_spin(bar(kBarRopeEmpty), (g - 1) & 1, abort_flag, a.status);
                    if (!ok) break;
                    if (leader) mbar_arrive_expect_tx(bar(kBarRopeFull), 2 * kSub);
                    tma_load_3d_pair(sb + kOffRope, &map_rope, 0, t.row, 8, lead(kBarRopeFull));
                }
                ++seg;
            }
        }
    } else if (!kFp8 && warp == 10) {
        // ------------------------------------------------ the other CTA's rows, this CTA's value columns
        if (lane == 0) {
            const int other = rank ^ 1;
            int g = 0, seg = 0;
            bool ok = true;
            for (; ok && pc.next(); ++seg) {
                const int32_t* tab = a.block_table + (int64_t)pc.b * a.max_blocks;
                int pb = half_block(a, tab, pc.n, pc.i0, other), pm = half_block(a, tab, pc.n, pc.i0, rank);
                for (int i = pc.i0; i < pc.i1; ++i, ++g) {
                    const HalfTile t = half_tile(a, pb, pc.n, i, other), mine = half_tile(a, pm, pc.n, i, rank);
                    if (i + 1 < pc.i1) {
                        pb = half_block(a, tab, pc.n, i + 1, other);
                        pm = half_block(a, tab, pc.n, i + 1, rank);
                    }
                    const bool tail = t.lim < kHalf || mine.lim < kHalf;
                    const int v = kBarV + (g & 1);
                    ok = mbar_wait_spin(bar(kBarS + (g & 1)), (g >> 1) & 1, abort_flag, a.status);
                    if (!ok) break;
                    if (tail) {
                        mbar_arrive_expect_tx(bar(kBarVTail + (g & 1)), 2 * kPair);
                        if (leader) mbar_arrive(bar(v));  // P's arrival covers these rows
                    } else if (leader) {
                        mbar_arrive_expect_tx(bar(v), 4 * kPair);
                    }
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t dst = pair_addr(entry_of(g, seg) + 2 * other + j);
                        if (tail)
                            tma_load_3d(dst, &map_pair, 0, t.row, 4 * rank + 2 * j, bar(kBarVTail + (g & 1)));
                        else
                            tma_load_3d_pair(dst, &map_pair, 0, t.row, 4 * rank + 2 * j, lead(v));
                    }
                }
            }
        }
    } else if (kFp8 && warp < 4 + kDequantWarps) {
        // ------------------------------------------------ FP8 entries, dequantised into the tiles
        auto dequantise = [&](auto two) {
        constexpr bool kTwo = decltype(two)::value;
        // A warp has 8 rows of every tile, a lane 16 codes (16 bytes) of a row at a time: fp16 code times fp16
        // scale; the scale's rounding is off by 2^-11, the product's by 2^-11 more.  A scale below fp16's normal
        // numbers (2^-14) would lose its bits: the codes of such a row are multiplied by 2^-14 first (exact) and then
        // by 2^14 scale.  Every row is multiplied twice, others by 1 first: without it 300 rows after 12,000
        // positions take 1,154 instead of 1,200 us, but with a branch around it 1,220 to 1,300.
        // Rows that take no part become zeros.
        // A turn has three stages: pairs 0..2 of tile g, the other CTA's rows of tile g - 1 (their slots are
        // free once S of that tile is done), pair 3 and the rotated values of tile g.  A stage's
        // registers are loaded again for the next turn as soon as they are stored, so that every load
        // has a turn to arrive.
        const int w = warp - 4, other = rank ^ 1;
        const int r8 = lane >> 2, q4 = lane & 3, row = w * 8 + r8, row4 = w * 8 + (lane >> 3);
        const uint8_t* pool = static_cast<const uint8_t*>(a.kv);
        auto wait = [&](int i, int parity) {
            if (ok) ok = wait_lanes(i < 0 ? 0u : bar(i), parity, lane, abort_flag, a.status);
        };
        const uint32_t s_row = sb + (uint32_t)row * 128u;
        const uint32_t g0 = (uint32_t)((2 * q4) ^ (row & 7)) << 4, g1 = (uint32_t)((2 * q4 + 1) ^ (row & 7)) << 4;
        // 2 x 16 codes of a group of 128 values to two tiles, `off` bytes into shared memory
        auto store32 = [&](const uint4& c0, const uint4& c1, float scale, uint32_t off) {
            const bool tiny = fabsf(scale) < 6.103515625e-5f;  // 2^-14
            const __half2 power = __float2half2_rn(tiny ? 6.103515625e-5f : 1.f);
            const __half2 factor = __float2half2_rn(tiny ? scale * 16384.f : scale);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint4& code = t ? c1 : c0;
                const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __half2_raw x =
                        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(cw[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
                    const __half2 y = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&x), power), factor);
                    o[e] = *reinterpret_cast<const uint32_t*>(&y);
                }
                st_shared_v4(s_row + off + t * kSub + g0, o[0], o[1], o[2], o[3]);
                st_shared_v4(s_row + off + t * kSub + g1, o[4], o[5], o[6], o[7]);
            }
        };
        // ... their low terms, what code * scale has beyond the value y that store32 makes of it: with f = fp16(scale) and
        // e = scale - f, code f - y is exact in a fused multiply-add and code e is added in another (e is kept 2^10
        // times larger and its code smaller, for fp16's smallest steps; a tiny scale is already 2^14 times larger).
        // With `first`, y goes to off_first.
        auto store32_low = [&](const uint4& c0, const uint4& c1, float scale, uint32_t off, uint32_t off_first, bool first) {
            const bool tiny = fabsf(scale) < 6.103515625e-5f;
            const float larger = tiny ? scale * 16384.f : scale;
            const __half2 power = __float2half2_rn(tiny ? 6.103515625e-5f : 1.f);
            const __half2 factor = __float2half2_rn(larger);
            const __half2 rest = __float2half2_rn((larger - __low2float(factor)) * (tiny ? 1.f : 1024.f));
            const __half2 smaller = __float2half2_rn(tiny ? 1.f : 9.765625e-4f);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint4& code = t ? c1 : c0;
                const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
                uint32_t o[8], o1[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __half2_raw x =
                        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(cw[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
                    const __half2 c = __hmul2(*reinterpret_cast<const __half2*>(&x), power), y = __hmul2(c, factor);
                    const __half2 low = __hfma2(__hmul2(c, smaller), rest, __hfma2(c, factor, __hneg2(y)));
                    o[e] = *reinterpret_cast<const uint32_t*>(&low);
                    o1[e] = *reinterpret_cast<const uint32_t*>(&y);
                }
                st_shared_v4(s_row + off + t * kSub + g0, o[0], o[1], o[2], o[3]);
                st_shared_v4(s_row + off + t * kSub + g1, o[4], o[5], o[6], o[7]);
                if (first) {
                    st_shared_v4(s_row + off_first + t * kSub + g0, o1[0], o1[1], o1[2], o1[3]);
                    st_shared_v4(s_row + off_first + t * kSub + g1, o1[4], o1[5], o1[6], o1[7]);
                }
            }
        };
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        uint4 kc[8], vc[4], rv[2];
        float4 ks;
        float2 vs;
        const uint32_t off_code = (uint32_t)row * kFp8EntryBytes + 16u * q4, off_scale = (uint32_t)row * kFp8EntryBytes + kFp8ScaleOff;
        const uint32_t off_rope = (uint32_t)row4 * kFp8EntryBytes + kFp8RopeOff + 16u * (lane & 7);
        auto first_entry = [&](int pool_row) { return pool + (int64_t)pool_row * kFp8EntryBytes; };
        auto load_k = [&](int pool_row, int lim) {  // tiles 0..5 and the scales
            const uint8_t* e = first_entry(pool_row);
            const bool in = row < lim;
#pragma unroll
            for (int c = 0; c < 6; ++c) kc[c] = in ? __ldg(reinterpret_cast<const uint4*>(e + off_code + 64 * c)) : zero;
            ks = in ? __ldg(reinterpret_cast<const float4*>(e + off_scale)) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        auto load_p3 = [&](int pool_row, int lim) {  // tiles 6 and 7, rotated values
            const uint8_t* e = first_entry(pool_row);
            const bool in = row < lim;
#pragma unroll
            for (int c = 6; c < 8; ++c) kc[c] = in ? __ldg(reinterpret_cast<const uint4*>(e + off_code + 64 * c)) : zero;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                rv[k] = row4 + 4 * k < lim ? __ldg(reinterpret_cast<const uint4*>(e + off_rope + 4 * k * kFp8EntryBytes)) : zero;
        };
        auto load_v = [&](int pool_row, int lim) {
            const uint8_t* e = first_entry(pool_row);
            const bool in = row < lim;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                vc[c] = in ? __ldg(reinterpret_cast<const uint4*>(e + off_code + 256 * rank + 64 * c)) : zero;
            vs = in ? __ldg(reinterpret_cast<const float2*>(e + off_scale + 8 * rank)) : make_float2(0.f, 0.f);
        };
        // the pair's tiles by turns, a piece after another: pool rows and limits of the next tile (my
        // rows, the other CTA's)
        int ti = 0, pm = -1, po = -1, m_row = 0, m_lim = 0, o_row = 0, o_lim = 0;
        const int32_t* tab = nullptr;
        auto next_tile = [&]() {
            if (ti >= pc.i1) {
                if (!pc.next()) return false;
                ti = pc.i0;
                tab = a.block_table + (int64_t)pc.b * a.max_blocks;
                pm = half_block(a, tab, pc.n, ti, rank);
                po = half_block(a, tab, pc.n, ti, other);
            }
            const HalfTile mine = half_tile(a, pm, pc.n, ti, rank), theirs = half_tile(a, po, pc.n, ti, other);
            if (mine.bad && w == 0 && lane == 0) record_status(a.status, DSA_STATUS_INDEX_OOB);
            m_row = mine.row, m_lim = mine.lim, o_row = theirs.row, o_lim = theirs.lim;
            ++ti;
            if (ti < pc.i1) {
                pm = half_block(a, tab, pc.n, ti, rank);
                po = half_block(a, tab, pc.n, ti, other);
            }
            return true;
        };
        auto publish = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
        };
        auto arrive = [&](int i) {
            if (ok && lane == 0) mbar_arrive_cluster(lead(i));
        };
        bool cur = next_tile(), prev = false;
        if (cur) {
            load_k(m_row, m_lim);
            load_p3(m_row, m_lim);
        }
        float ks3 = 0.f;
        int slot = 0, use = 0;   // ring slot of the tile's pair 0, and how often the ring has gone round there
        uint32_t v_off = 0;      // the tile before: slot of the other rows' first pair
        int v_slot1 = 0;
        auto advance = [&]() {
            slot += 4;
            if (slot >= kRing) {
                slot -= kRing;
                ++use;
            }
        };
        for (int g = 0; ok && (cur || prev); ++g) {
            bool nxt = false;
            int s[4];
            auto next_slots = [&]() {
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = slot + j >= kRing ? slot + j - kRing : slot + j;
            };
            next_slots();
            const int r_row = o_row, r_lim = o_lim;  // the other CTA's rows of tile g
            if (cur) {
                nxt = next_tile();
                ks3 = ks.w;
                if constexpr (kTwo) {  // the low terms' entries, then pairs 0..2
                    const bool wrap = slot + lane >= kRing;
                    wait(lane < 7 && use + (wrap ? 1 : 0) > 0 ? kBarPairEmpty + slot + lane - (wrap ? kRing : 0) : -1,
                         (use + (wrap ? 0 : 1)) & 1);
                    const int low[4] = {s[0], s[1], s[2], s[3]};
                    advance();
                    next_slots();
                    if (ok) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            store32_low(kc[2 * j], kc[2 * j + 1], j == 0 ? ks.x : j == 1 ? ks.y : j == 2 ? ks.z : ks.w, low[j] * kPair,
                                        s[j] * kPair, j < 3);
                    }
                    publish();
#pragma unroll
                    for (int j = 0; j < 4; ++j) arrive(kBarPairFull + low[j]);
#pragma unroll
                    for (int j = 0; j < 3; ++j) arrive(kBarPairFull + s[j]);
                } else {
                    const bool wrap = slot + lane >= kRing;
                    wait(lane < 3 && use + (wrap ? 1 : 0) > 0 ? kBarPairEmpty + slot + lane - (wrap ? kRing : 0) : -1,
                         (use + (wrap ? 0 : 1)) & 1);
                    if (ok) {
#pragma unroll
                        for (int j = 0; j < 3; ++j)
                            store32(kc[2 * j], kc[2 * j + 1], j == 0 ? ks.x : j == 1 ? ks.y : ks.z, s[j] * kPair);
                    }
                    publish();
#pragma unroll
                    for (int j = 0; j < 3; ++j) arrive(kBarPairFull + s[j]);
                }
                if (nxt) load_k(m_row, m_lim);
            }
            if (prev) {
                wait(kBarS + ((g - 1) & 1), ((g - 1) >> 1) & 1);
                if (ok) {
                    store32(vc[0], vc[1], vs.x, v_off);
                    store32(vc[2], vc[3], vs.y, v_slot1 * kPair);
                }
                publish();
                arrive(kBarV + ((g - 1) & 1));
            }
            if (cur) {
                load_v(r_row, r_lim);
                {
                    const int round = use + (slot + 3 >= kRing ? 1 : 0);
                    wait(lane == 0 && round > 0 ? kBarPairEmpty + s[3] : lane == 1 && g > 0 ? kBarRopeEmpty : -1,
                         lane == 0 ? (round + 1) & 1 : (g + 1) & 1);
                }
                if (ok) {
                    store32(kc[6], kc[7], ks3, s[3] * kPair);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int rr = row4 + 4 * k;
                        st_shared_v4(sb + kOffRope + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4), bf16x2_to_f16x2(rv[k].x),
                                     bf16x2_to_f16x2(rv[k].y), bf16x2_to_f16x2(rv[k].z), bf16x2_to_f16x2(rv[k].w));
                    }
                }
                publish();
                arrive(kBarPairFull + s[3]);
                arrive(kBarRopeFull);
                if (nxt) load_p3(m_row, m_lim);
            }
            v_off = (other ? s[2] : s[0]) * kPair;
            v_slot1 = other ? s[3] : s[1];
            advance();
            prev = cur;
            cur = nxt;
        }
        };
        if (pc.two)  // (the same for the whole pair)
            dequantise(std::true_type{});
        else if constexpr (kMixed)
            dequantise(std::false_type{});
    } else {
        // the issuing warp; over FP8 entries its warpgroup, whose four warps execute the one instruction that gives
        // registers back (three of them have nothing else to do)
        if constexpr (kFp8) setmaxnreg_dec<kRegsIssue>();
        if (leader && warp == kMmaWarp) {
        auto issue = [&](auto two) {
        constexpr bool kTwo = decltype(two)::value;
        // ------------------------------------------------ MMA issue (converged warp, one elected lane)
        // Order: Q K^T of a tile, then P V of the tile before, so that the softmax of one tile overlaps
        // the products of its neighbours; where a new row begins P V goes first (the row's query block
        // is still on its way).  All barriers that a step needs are polled at once, one a lane.
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t s0 = __shfl_sync(0xffffffffu, sb, 0);
        const uint64_t d_k = make_smem_desc(s0 + kOffRing, 16, 1024, kSwizzle128B);
        const uint64_t d_rope = make_smem_desc(s0 + kOffRope, 16, 1024, kSwizzle128B);
        const uint64_t d_q = make_smem_desc(s0 + kOffQ, 16, 1024, kSwizzle128B);
        const uint64_t d_p = make_smem_desc(s0 + kOffP, 16, 1024, kSwizzle128B);
        const uint64_t d_v = make_smem_desc(s0 + kOffRing, kSub, 1024, kSwizzle128B);
        bool ok = true;
        auto wait_all = [&](int i, int parity) {
            if (ok) ok = wait_lanes(i < 0 ? 0u : bar(i), parity, lane, abort_flag, a.status);
            tc_fence_after();
        };
        auto issue_pv = [&](int g, bool first, int seg) {
            const int i = lane == 0 ? kBarP : lane == 1 ? kBarV + (g & 1) : lane == 2 && first && seg > 0 ? kBarOFree : -1;
            wait_all(i, lane == 0 ? g & 1 : lane == 1 ? (g >> 1) & 1 : (seg - 1) & 1);
            if (ok && elect_one()) {
                int slot = entry_of(g, seg, kTwo) % kRing;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int vh = 0; vh < 2; ++vh) {
                        const uint32_t off = (uint32_t)slot * kPair;
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_pair_f16_ss(tm + 128u * vh, d_p + ((x * kSub + ks * 32) >> 4), d_v + ((off + ks * 2048) >> 4),
                                            kIdescPV, (x == 0 && ks == 0) ? (first ? 0u : 1u) : 1u);
                        mma_pair_commit(bar(kBarPairEmpty + slot));
                        if (++slot == kRing) slot = 0;
                    }
                }
                mma_pair_commit(bar(kBarO));
            }
            __syncwarp();
        };
        int g = 0, seg = 0;
        bool pv_first = false;  // the tile before g began its row
        while (ok && pc.next()) {
            const int n = pc.i1 - pc.i0;
            for (int t = 0; t < n && ok; ++t, ++g) {
                if (t == 0 && g > 0) issue_pv(g - 1, pv_first, seg - 1);
                const int entry = entry_of(g, seg, kTwo);
                if (kTwo) {
                    const int p = entry - 4 + lane;
                    const int i = lane < 4 ? kBarPairFull + p % kRing : lane == 4 && t == 0 ? kBarQ : lane == 5 && g > 0 ? kBarSFree : -1;
                    wait_all(i, lane < 4 ? (p / kRing) & 1 : lane == 4 ? seg & 1 : (g - 1) & 1);
                    if (ok && elect_one()) {
                        int s = (entry - 4) % kRing;
#pragma unroll 1
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t off = (uint32_t)s * kPair;
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const uint64_t b = d_k + ((off + (c >> 2) * kSub + (c & 3) * 32) >> 4);
                                if (j < kQTmem / 2)
                                    mma_pair_f16_ts(tm + kColS, tm + kColQ + 64u * j + 8u * c, b, kIdescQK, (j | c) ? 1u : 0u);
                                else
                                    mma_pair_f16_ss(tm + kColS, d_q + (((c >> 2) * kSub + (c & 3) * 32) >> 4), b, kIdescQK, 1u);
                            }
                            mma_pair_commit(bar(kBarPairEmpty + s));
                            if (++s == kRing) s = 0;
                        }
                    }
                    __syncwarp();
                    // (the ring has no room for two whole tiles and low terms: P V before the tile's own products)
                    if (t > 0) issue_pv(g - 1, t == 1, seg);
                }
                {
                    // pairs 0..2, S, and where a piece begins its query tiles (lanes 5..7: their ring entries)
                    const int p = entry + (lane < 3 ? lane : lane - 5 - kQEntries);
                    const int i = lane < 3 || (!kFp8 && t == 0 && lane >= 5 && lane < 5 + kQEntries) ? kBarPairFull + p % kRing
                                  : lane == 3 && g > 0 ? kBarSFree
                                  : kFp8 && lane == 4 && t == 0 ? kBarQ : -1;
                    wait_all(i, lane == 3 ? (g - 1) & 1 : lane == 4 ? seg & 1 : (p / kRing) & 1);
                }
                if (!kFp8 && t == 0 && ok && elect_one()) {
                    // (the piece before's Q K^T are complete: its S has been read)
#pragma unroll 1
                    for (int j = 0; j < kQEntries; ++j) {
                        const int slot = (entry - kQEntries + j) % kRing;
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            tmem_copy_pair_64x128b(tm + kColQ + 64u * j + 4u * c,
                                                   d_k + ((slot * kPair + (c >> 3) * kSub + (c & 7) * 16) >> 4));
                        mma_pair_commit(bar(kBarPairEmpty + slot));
                    }
                }
                __syncwarp();
                if (ok && elect_one()) {
                    int s = entry % kRing;
#pragma unroll
                    for (int j = 0; j < kQTmem / 2; ++j) {
                        const uint32_t off = (uint32_t)s * kPair;
#pragma unroll
                        for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_pair_f16_ts(tm + kColS, tm + kColQ + 32u * (2 * j + cc) + 8u * kk,
                                                d_k + ((off + cc * kSub + kk * 32) >> 4), kIdescQK, kTwo || (j | cc | kk) ? 1u : 0u);
                        if (++s == kRing) s = 0;
                    }
                }
                __syncwarp();
                {
                    const int p = entry + 3;
                    wait_all(lane == 0 ? kBarPairFull + p % kRing
                             : lane == 1 ? kBarRopeFull
                             : !kFp8 && lane == 2 && t == 0 ? kBarQ : -1,
                             lane == 0 ? (p / kRing) & 1 : lane == 1 ? g & 1 : seg & 1);
                }
                if (ok && elect_one()) {
                    const uint32_t off = (uint32_t)((entry + 3) % kRing) * kPair;
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_pair_f16_ss(tm + kColS, d_q + ((cc * kSub + kk * 32) >> 4),
                                            d_k + ((off + cc * kSub + kk * 32) >> 4), kIdescQK, 1u);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_pair_f16_ss(tm + kColS, d_q + ((2 * kSub + kk * 32) >> 4), d_rope + ((kk * 32) >> 4), kIdescQK, 1u);
                    mma_pair_commit(bar(kBarS + (g & 1)));
                    mma_pair_commit(bar(kBarRopeEmpty));
                    if (t + 1 == n) mma_pair_commit(bar(kBarQFree));
                }
                __syncwarp();
                if (t > 0 && !kTwo) issue_pv(g - 1, t == 1, seg);
            }
            pv_first = n == 1;
            ++seg;
        }
        if (ok && g > 0) issue_pv(g - 1, pv_first, seg - 1);
        };
        if (pc.two)
            issue(std::bool_constant<kFp8>{});
        else if constexpr (kMixed || !kFp8)
            issue(std::false_type{});
        }
    }
}

template <bool kFp8, bool kMixed>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFp8 ? kThreadsFp8 : kThreadsBf16, 1)
    chunk_attn_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap map_pair,
                      const __grid_constant__ CUtensorMap map_rope, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_q3) {
    constexpr int kThreads = kFp8 ? kThreadsFp8 : kThreadsBf16;
    constexpr int kWarps = kThreads / 32;
    constexpr int kMmaWarp = kFp8 ? 12 : 9;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    if ((sb & 1023u) != 0) {  // the declared alignment holds: no other shared memory precedes it
        record_status(a.status, DSA_STATUS_INVALID_ARG);
        return;
    }
    Shared* sh = reinterpret_cast<Shared*>(smem + kOffMisc);
    volatile int* abort_flag = &sh->abort_flag;
    auto bar = [&](int i) { return sb + kOffBar + 8u * i; };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = blockIdx.x >> 1;

    if (tid == 0) {
        // filled by TMA (the leader's expected bytes) or by both CTAs' dequantising warps
        constexpr int kFill = kFp8 ? 2 * kDequantWarps : 1;
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar(kBarPairFull + i), kFill);
            mbar_init(bar(kBarPairEmpty + i), 1);
        }
        mbar_init(bar(kBarRopeFull), kFill);
        mbar_init(bar(kBarRopeEmpty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarV + i), kFill);
            mbar_init(bar(kBarVTail + i), 1);
            mbar_init(bar(kBarS + i), 1);
            mbar_init(bar(kBarStat + i), 4);  // a softmax warp each
        }
        mbar_init(bar(kBarSFree), 8);   // a softmax warp each, both CTAs
        mbar_init(bar(kBarP), 8);
        mbar_init(bar(kBarO), 1);
        mbar_init(bar(kBarOFree), 8);
        mbar_init(bar(kBarQ), kFp8 ? 8 : 1);  // a query warp each, both CTAs; or the leader's expected bytes
        mbar_init(bar(kBarQFree), 1);
        sh->abort_flag = 0;
        sh->row0 = sh->skip = sh->count = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(smem_u32(&sh->tmem_base), 512);
        tmem_relinquish_pair();
    }

    griddep_wait();  // (the lengths may come from the kernel before)

    // ---- the plan: this pair's piece [lo, hi) of the line of all rows' units
    bool empty_rows = false;
    {
        // (kMixed: two lines, of the rows with two terms and of the others, each with pairs of its own)
        constexpr int kKinds = kMixed ? 2 : 1;
        long long (*sums)[kMaxWarps] = reinterpret_cast<long long (*)[kMaxWarps]>(smem + kOffMax);  // (not in use yet)
        const int per = (a.Nq + kThreads - 1) / kThreads;
        const int t0 = tid * per, t1 = min(a.Nq, t0 + per);
        long long mine[kKinds] = {}, incl[kKinds];
        for (int t = t0; t < t1; ++t) {
            const int n = __ldg(a.q_len + t), b = __ldg(a.q_seq + t);
            const int k = tiles_of(a, n, b);
            const bool one = kMixed && !two_terms(n);  // (selected: an index would put the sums into local memory)
            mine[0] += one ? 0 : units_of(k);
            mine[kKinds - 1] += one ? units_of(k) : 0;
            empty_rows |= k == 0;
            if (blockIdx.x == 0 && !row_ok(a, n, b)) record_status(a.status, DSA_STATUS_LENGTH);
        }
#pragma unroll
        for (int x = 0; x < kKinds; ++x) {
            incl[x] = mine[x];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, incl[x], o);
                if (lane >= o) incl[x] += v;
            }
            if (lane == 31) sums[x][warp] = incl[x];
        }
        empty_rows = __syncthreads_or(empty_rows);
        long long before[kKinds] = {}, sum[kKinds] = {};
        for (int w = 0; w < kWarps; ++w) {
#pragma unroll
            for (int x = 0; x < kKinds; ++x) {
                if (w < warp) before[x] += sums[x][w];
                sum[x] += sums[x][w];
            }
        }
        // this pair's kind, and its place among the pairs of that kind: pairs as the kinds' work, one at least each
        int kind = 0, base = 0, pairs = a.clusters;
        if constexpr (kMixed) {
            const long long cost = kTwoCost * sum[0], both = cost + kOneCost * sum[1];
            const int first = sum[0] == 0 ? 0 : sum[1] == 0 ? a.clusters
                              : (int)min(max((a.clusters * cost + both / 2) / both, 1ll), a.clusters - 1ll);
            kind = cluster >= first;
            base = kind ? first : 0;
            pairs = kind ? a.clusters - first : first;
        }
        const bool other = kMixed && kind == 1;
        const long long total = other ? sum[kKinds - 1] : sum[0], units = other ? mine[kKinds - 1] : mine[0];
        long long at = (other ? before[kKinds - 1] + incl[kKinds - 1] : before[0] + incl[0]) - units;
        const int place = cluster - base;
        // (a row's pieces are consecutive pairs': a pair between its first and its last has units of its tiles)
        const long long most = total < 16ll * a.Nq ? total : max(16ll, total / min_piece<kFp8>());
        const int pieces = (int)min((long long)pairs, most);
        const long long lo = place < pieces ? total * place / pieces : total;
        const long long hi = place < pieces ? total * (place + 1) / pieces : total;
        if (tid == 0) {
            sh->pieces = pieces;
            sh->base = base;
            sh->two = kind == 0;
            sh->lo = lo;
            sh->total = total;
            sh->count = (int)(hi - lo);
        }
        if (hi > lo && at <= lo && lo < at + units) {
            for (int t = t0; t < t1; ++t) {
                const int n = __ldg(a.q_len + t);
                if (kMixed && two_terms(n) != (kind == 0)) continue;
                const int k = units_of(tiles_of(a, n, __ldg(a.q_seq + t)));
                if (lo < at + k) {
                    sh->row0 = t;
                    sh->skip = (int)(lo - at);
                    break;
                }
                at += k;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();

    chunk_roles<kFp8, kMixed>(a, map_pair, map_rope, map_q, map_q3, sb, sh, empty_rows);

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a wait ran out: what this CTA still has in flight lands before its memory goes away
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    __syncwarp();
    cluster_sync_all();
    griddep_launch_dependents();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair((uint32_t)sh->tmem_base, 512);
    }
}

// Merge of the rows that cross pieces: O = sum_p exp(lse_p - L) O_p / sum_p exp(lse_p - L) over the
// pieces in the order of their positions.  Every CTA lists the rows that start in one pair and end in
// another, and takes its share of units: of a row of few pieces four heads, one a warp; of a row of many
// (one long row over 74 pairs is 128 heads x 74 x 2 KB) half of a head, whose pieces its four warps share.
constexpr int kMaxClusters = 128;
// Five CTAs of 96 registers a thread fit an SM and are launched (measured: eight of 64 registers spill and cost a
// 64-row decode 80 instead of 62 us; eight warps a CTA, a head each, 66 us).
constexpr int kMergeWarps = 4, kMergeCtasPerSm = 5;
constexpr int kMergeShared = 8;  // pieces from which a head is shared by warps

// One warp: pieces p0, p0 + step, .. of head h, values 128 q + 4 lane .. + 3 of its kQ x 128; the sum of
// the weighted pieces, and L and the weights' sum.
template <int kQ>
__device__ __forceinline__ void merge_pieces(const ChunkArgs& a, const int4& m, int h, int at, int p0, int step, int lane,
                                             float4 (&acc)[kQ], float& L, float& sum) {
    constexpr int kDeep = 8 / kQ;  // pieces in flight
    const int np = m.w;
    auto slot_of = [&](int p) { return p == 0 ? m.y : 2 * (m.z + p); };
    const float4* part = reinterpret_cast<const float4*>(a.part_o) + (int64_t)h * (kDV / 4) + at + lane;
    float4 v[kDeep][kQ];
    auto fetch = [&](int p) {
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                if (p + k * step < np) v[k][q] = part[(int64_t)slot_of(p + k * step) * (kMlaHeads * kDV / 4) + 32 * q];
    };
    fetch(p0);  // on their way while the weights are made
    float ls[kMaxClusters / 32];
    L = -CUDART_INF_F;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxClusters / 32; ++k) {
        ls[k] = lane + 32 * k < np ? a.part_lse[slot_of(lane + 32 * k) * kMlaHeads + h] : -CUDART_INF_F;
        L = fmaxf(L, ls[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, o));
#pragma unroll
    for (int k = 0; k < kMaxClusters / 32; ++k) {
        ls[k] = ls[k] == -CUDART_INF_F ? 0.f : __expf(ls[k] - L);
        sum += ls[k];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int q = 0; q < kQ; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = p0; p < np; p += kDeep * step) {
        if (p != p0) fetch(p);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int i = p + k * step;
            if (i >= np) break;  // (the same for the whole warp)
            const float x = i < 32 ? ls[0] : i < 64 ? ls[1] : i < 96 ? ls[2] : ls[3];
            const float e = __shfl_sync(0xffffffffu, x, i & 31);
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                acc[q].x = fmaf(e, v[k][q].x, acc[q].x);
                acc[q].y = fmaf(e, v[k][q].y, acc[q].y);
                acc[q].z = fmaf(e, v[k][q].z, acc[q].z);
                acc[q].w = fmaf(e, v[k][q].w, acc[q].w);
            }
        }
    }
}

__global__ void __launch_bounds__(32 * kMergeWarps, kMergeCtasPerSm) chunk_combine_kernel(const ChunkArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ int4 rows[kMaxClusters];      // row, first piece's slot, first pair, pieces
    __shared__ int first[kMaxClusters + 1];  // first unit
    __shared__ float4 part_sum[kMergeWarps][kDV / 8];
    __shared__ int nrows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {
        int4 meta[kMaxClusters / 32];
#pragma unroll
        for (int k = 0; k < kMaxClusters / 32; ++k)
            meta[k] = lane + 32 * k < a.clusters ? a.meta[lane + 32 * k] : make_int4(-1, 0, 0, 0);
        int n = 0, units = 0;
#pragma unroll
        for (int k = 0; k < kMaxClusters / 32; ++k) {
            const bool have = meta[k].x >= 0;
            const unsigned mask = __ballot_sync(0xffffffffu, have);
            if (mask == 0) continue;
            const int c = lane + 32 * k, np = meta[k].z - c + 1;
            const int mine = have ? (np >= kMergeShared ? 2 * kMlaHeads : kMlaHeads / kMergeWarps) : 0;
            int before = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += v;
            }
            if (have) {
                const int i = n + __popc(mask & ((1u << lane) - 1));
                rows[i] = make_int4(meta[k].x, meta[k].y, c, np);
                first[i] = units + before - mine;
            }
            n += __popc(mask);
            units += __shfl_sync(0xffffffffu, before, 31);
        }
        if (lane == 0) {
            first[n] = units;
            nrows = n;
        }
    }
    __syncthreads();
    const int total = first[nrows];
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
        int lo = 0, hi = nrows - 1;  // the last row whose first unit is at most u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int4 m = rows[lo];
        const int i = u - first[lo];
        const bool shared = m.w >= kMergeShared;
        const int h = shared ? i >> 1 : i * kMergeWarps + warp;
        float L, sum;
        uint2* out = reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + ((int64_t)m.x * kMlaHeads + h) * kDV);
        auto put = [&](int at, const float4& x) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            out[at] = make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
        };
        if (!shared) {
            float4 acc[4];
            merge_pieces(a, m, h, 0, 0, 1, lane, acc, L, sum);
#pragma unroll
            for (int q = 0; q < 4; ++q) put(lane + 32 * q, acc[q]);
        } else {
            float4 acc[2];
            const int at = (i & 1) * (kDV / 8);
            merge_pieces(a, m, h, at, warp, kMergeWarps, lane, acc, L, sum);
#pragma unroll
            for (int q = 0; q < 2; ++q) part_sum[warp][lane + 32 * q] = acc[q];
            __syncthreads();
            if (threadIdx.x < kDV / 8) {
                float4 x = part_sum[0][threadIdx.x];
#pragma unroll
                for (int k = 1; k < kMergeWarps; ++k) {
                    const float4 y = part_sum[k][threadIdx.x];
                    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                }
                put(at + threadIdx.x, x);
            }
            __syncthreads();
        }
        if (lane == 0 && a.lse && (!shared || (warp == 0 && (i & 1) == 0)))
            a.lse[(int64_t)m.x * kMlaHeads + h] = sum == 0.f ? -CUDART_INF_F : L + __logf(sum);
    }
}

}  // namespace

cudaError_t launch_chunk_attn(const ChunkArgs& a, cudaStream_t st) {
    if (a.Nq == 0) return cudaSuccess;
    if (a.clusters < 1 || a.clusters > kMaxClusters) return cudaErrorInvalidValue;
    alignas(64) CUtensorMap mp = {}, mr = {}, mq = {}, m3 = {};  // over FP8 entries everything is read by plain loads
    const uint64_t rows = (uint64_t)a.num_blocks << a.block_shift;
    if (!a.kv_fp8 && (!encode_tensor_map_rows_bf16(&mp, a.kv, rows, kDK / 64, kHalf, 2) ||
                      !encode_tensor_map_rows_bf16(&mr, a.kv, rows, kDK / 64, kHalf, 1) ||
                      !encode_tensor_map_rows_bf16(&mq, a.q, (uint64_t)a.Nq * kMlaHeads, kDK / 64, kHeads, 2) ||
                      !encode_tensor_map_rows_bf16(&m3, a.q, (uint64_t)a.Nq * kMlaHeads, kDK / 64, kHeads, 3)))
        return cudaErrorInvalidValue;
    using Kernel = void (*)(ChunkArgs, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap);
    static constexpr Kernel kernels[3] = {chunk_attn_kernel<false, false>, chunk_attn_kernel<true, false>, chunk_attn_kernel<true, true>};
    // (a table of up to kTwoTerms positions has rows with two terms only)
    const int kind = !a.kv_fp8 ? 0 : a.T_max > kTwoTerms ? 2 : 1;
    // the shared-memory limit is a setting of the kernel on a device: raised once each
    static std::atomic<bool> raised[3][kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (!known || !raised[kind][dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernels[kind], cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        if (known) raised[kind][dev].store(true, std::memory_order_release);
    }
    // both kernels may be set up while the one before them still runs; they wait for it on the device
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = st;
    cfg.gridDim = dim3(2 * a.clusters, 1, 1);
    cfg.blockDim = dim3(a.kv_fp8 ? kThreadsFp8 : kThreadsBf16, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    e = cudaLaunchKernelEx(&cfg, kernels[kind], a, mp, mr, mq, m3);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * a.clusters * kMergeCtasPerSm, 1, 1);
    cfg.blockDim = dim3(32 * kMergeWarps, 1, 1);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, chunk_combine_kernel, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace dsa
