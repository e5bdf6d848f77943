// attention_chunk.cuh -- attention of many query rows per KV head (prefill
// chunks, wide verifies) over the quantised paged cache, on tcgen05.
//
// With n new tokens and G query heads per KV head every cached element is used by
// n * G rows, so the two products bound the kernel.  What a score costs beside
// them (read from tensor memory, scaled, 2^x, summed, rounded to f16, stored) is
// half as much again for the warps that do it.  One CTA per SM, two row tiles of
// 128 in flight so that the tensor pipe works on one while the other is in its
// softmax; warps by role:
//
//   warps 0-3, 4-7  softmax of row tile 0 and 1: a thread has one row.  Scores
//                   come from tensor memory and the weights P go back there as
//                   the f16 A operand of the second product, over the scores.
//   warps 18, 19    bulk copies of K's, and V's, codes, scales and exponents from
//                   the pages to shared memory, ahead of their conversion.
//   warps 8-11, 12-15  codes of K, and of V, to f16, from there to the layout of the MMA's B operands
//                   (K with the head dimension contiguous; V likewise, read
//                   transposed).
//   warps 16, 17    MMA issue for row tile 0 and 1: S = Q K^T, O += P V.
//
// The roles share one instruction cache: each one's loop is kept short (half a
// tile's scores at a time, one loop body for K and V), because straight-line
// code for whole tiles, with variants for masked ones, ran out of it.
//
// SPLIT: when a sequence has at most 128 rows, both softmax groups take the same
// row tile, one the even and the other the odd key tiles, and their results
// are joined at the end; otherwise half the pipeline would idle.
//
// f16 holds codes exactly.  A row's power of two is applied relative to a unit of
// its tile of 128 keys, that of the largest row, whose exponent goes to the softmax
// as one factor (K) and one addend (V; see attention_decode.cuh).  That is exact
// while no row lies more than 2^14 (kBelow) below the unit.  V's unit also sets
// what the f16 weights of other tiles lose (for a row of Q, relative to the largest
// unit beside its largest weight), so a key that a row does not see must not raise
// it: in tiles whose keys some rows see and others do not, the unit is that of the
// largest row that all see (or of the smallest, if all see none), as far as f16 holds
// the others' codes times up to kAbove.  2^6 (kUnseen) more than that makes the
// weights' loss 2^-24 per key where it was 2^-28; ordinary V rows need it, where no key of
// a tile is seen by all (one query head per KV head, NVFP4).  A tile that
// breaks these rules is left out (its pages count as not there), and a segment that had
// one adds such tiles at its end, in fp32 and with each key's exponents apart
// (far_tiles).  (A loop of its own for them among the softmax warps' tiles took up to
// 20 % of a long chunk's time even where no tile was one: the roles' loops fill the
// instruction cache, and the checks alone take 5 %.  A second launch of the few-row kernel, which ended at once
// where there was none, took 2 to 3 us a call.)  Outputs are bf16 only.
//
// A tile's scores are made in two halves of 64 keys, each in columns of its own,
// which its weights then take: the next half's scores are made while the
// softmax is at this one.  A row's reference (an upper estimate of its largest
// score) moves only when the weights of a half sum to more than 2^15, so there is
// no pass for the maximum.
//
// Measured on one GB300: 2048 tokens behind 14336 cached ones (E4M3, 40 and 8 heads
// of 128, 644 GFLOP) 550 us, 1.17 PFLOP/s, 0.60 of the measured bf16 rate;
// 2 x 512 tokens in a window of 4096 101 us; 8 trees of 16 tokens over 2016 to
// 6017 NVFP4 keys 37.9 us; four ragged prefills of up to 1500 tokens (heads of 64,
// NVFP4) 41.9 us.  A tile of 256 rows and 128 keys takes about 4200 clocks,
// 3300 of them the softmax warps' own chain; the MMAs alone would take 2600.
#pragma once

#include <cstdint>

#include "attention_ops.cuh"
#include "attention_plan.cuh"
#include "skinny.cuh"

namespace nvfp4 {
namespace attn {
namespace chunk {

constexpr int kTile = 128;                      // keys of a tile
constexpr int kRowTile = 128;                   // rows of a row tile
constexpr int kSoftmaxWarps = 8, kConvertWarps = 8;
constexpr int kConvertThreads = 32 * kConvertWarps / 2;  // of K, and as many of V
constexpr int kThreads = 32 * (kSoftmaxWarps + kConvertWarps + 4);  
// Registers of a thread by role: what the launch gives every thread, shared out anew.
constexpr int kSoftmaxRegs = 128, kConvertRegs = 72, kMmaRegs = 72, kLaunchRegs = 96;
static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kConvertWarps * kConvertRegs + 4 * kMmaRegs) <= kThreads * kLaunchRegs,
              "setmaxnreg would wait for registers that nobody gives back");
constexpr int kStages = 2;
constexpr int kInfos = 4;
constexpr int kMostRaw = 4;         // buffers of K or V as they lie in the pages
constexpr int kSharedBytes = 1024;  // barriers and the like (Shared)
// What an item costs a CTA beside its tiles, in tiles.  (Ragged prefill of four sequences: 61.1 us at 0, 40.8 at 2,
// 41.2 at 3, 43.7 at 8; 8 trees of 16 tokens 37.8, 35.8, 35.4, 35.4.)
constexpr int kItemCost = 3;
constexpr int kBelow = 14, kUnseen = 6;
constexpr int kNear = 48;  // of V's units, for the softmax sums (attention_decode.cuh)
constexpr float kHeadroom = 7.f;
constexpr float kMostWeight = 0x1p15f;  // of the weights of half a tile, in sum
constexpr float kSumUnit = 0x1p-32f;

// Codes of the status word (waits that ran out).
enum : uint32_t { kTimeoutSoftmax = 51, kTimeoutConvert = 52, kTimeoutMma = 53, kTimeoutLoad = 54 };

template <int FMT, int D, bool SPLIT>
struct Cfg {
    using R = kv::Row<FMT, D>;
    static constexpr int kRows = SPLIT ? kRowTile : 2 * kRowTile;
    static constexpr int kOperand = 128 * D * 2;  // Q, K or V tile in f16
    static constexpr int kQAt = 0, kKAt = (SPLIT ? 1 : 2) * kOperand, kVAt = kKAt + kStages * kOperand;
    // a tile's bytes as they lie in the pages, run by run (codes, scales, exponents); K's with V's exponents behind.
    // One tile's loads take as long as its conversion, so there are as many buffers as fit, for K first.
    static constexpr int kRawRows = kTile * R::kBytes;
    static constexpr int kRawKBytes = kRawRows + kTile, kRawVBytes = kRawRows;
    static constexpr int kStatsBytes = SPLIT ? 2 * kRowTile * 8 : 0;
    static constexpr int kRawAt = kVAt + kStages * kOperand;
    static constexpr int kRoom = 227 * 1024 - kRawAt - kStatsBytes - kSharedBytes;
    static constexpr int kRawPairs = kRoom / (kRawKBytes + kRawVBytes);
    static constexpr int kRawVs = kRawPairs < kMostRaw ? kRawPairs : kMostRaw;
    static constexpr int kRawKs = kRawVs < kMostRaw && kRoom - kRawVs * (kRawKBytes + kRawVBytes) >= kRawKBytes ? kRawVs + 1 : kRawVs;
    static constexpr int kRawKAt = kRawAt, kRawVAt = kRawKAt + kRawKs * kRawKBytes;
    static constexpr int kStatsAt = kRawVAt + kRawVs * kRawVBytes;
    static constexpr int kBarAt = kStatsAt + kStatsBytes;
    static constexpr int kSmem = kBarAt + kSharedBytes;
    static_assert(kRawVs >= 1, "shared memory");
    static constexpr int kSlotFloats = kRows * (D + 2);
    // tensor memory columns
    static constexpr int kScoreCols = 0, kOutCols = 2 * kTile;
    // log2 of how far a row of V may exceed its tile's unit: 448 * 2^7 and 2688 * 2^4 are f16 numbers
    static constexpr int kAbove = FMT == NVFP4_KV_E4M3 ? 7 : 4;
    // 16-byte chunks of codes of a 64-element column block of a row.  A thread's lie in kRowsMine rows, kRowStep apart.
    static constexpr int kPerBlock = FMT == NVFP4_KV_E4M3 ? 4 : 2;
    static constexpr int kRowStep = kConvertThreads / kPerBlock, kRowsMine = kTile / kRowStep;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// What a converted tile tells the softmax.
struct TileInfo {
    float k_unit;      // 2^(exponent of K's unit)
    float v_exp;       // exponent of V's unit
    uint32_t present;  // bit g: the page of keys 16 g .. 16 g + 15 is there, or no row sees them
    uint32_t pad;
};

// Where the tile in the raw buffers lies.
struct RawInfo {
    int key0, lo, hi;
    int all_lo, all_hi;  // keys that every row of the item sees
    uint32_t present;

    // whether some row does not see some key of the tile that another one may see
    NVFP4_DEVINL bool mixed() const { return max(key0, lo) < all_lo || min(key0 + kTile, hi) > all_hi; }
};

// The part of an item that a CTA works on: the softmax warps' place in the CTA's range.
struct Segment {
    Item it;
    int64_t item_begin;  // first place of the item in the call's list
    int64_t u;           // place of the first tile
    int32_t tile0, n;    // first key tile, and number of tiles (0: none left)
    uint32_t index;                // of the first tile among the CTA's
};

struct Shared {
    uint64_t raw_full[2][kMostRaw], raw_empty[2][kMostRaw];  // K's, V's
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t q_ready[2], s_full[2][2], p_ready[2][2], pv_done[2][2], drain[2];  // by group, and half of the keys
    TileInfo info[kInfos];
    RawInfo raw[2][kMostRaw];
    Segment seg;
    uint32_t tmem, last, tiles;
    uint32_t far_tile;  // the last tile of the CTA whose rows lie far from its units, counted from 1
    int64_t scratch[kThreads / 32 + 5];
};
static_assert(sizeof(Shared) <= kSharedBytes, "barriers");

// Address of 16-byte chunk `oc` (8 elements) of row `r` of a 128-row f16
// operand: 64-element column blocks of 128 rows x 128 bytes, chunks of a row
// permuted by the 128-byte swizzle.
NVFP4_DEVINL uint32_t operand_chunk(uint32_t base, int r, int oc)
{
    return base + (oc >> 3) * (128 * 128) + r * 128 + (((oc & 7) ^ (r & 7)) << 4);
}

// A softmax group's part of a tile's sequence: with SPLIT, group g takes the
// tiles of an item whose index in the CTA's list has parity g.
template <bool SPLIT>
NVFP4_DEVINL bool takes(int group, uint32_t tile) { return !SPLIT || (tile & 1) == (uint32_t)group; }

// Whether a segment of n tiles from `tile` on has any for the group.
template <bool SPLIT>
NVFP4_DEVINL bool has_tile(int group, uint32_t tile, int n) { return n >= 2 || takes<SPLIT>(group, tile); }

// Moves place u of a CTA's range, which lies in the item or at its end, on to the
// next place with a tile (an item's first c.item_cost places have none), into
// the items behind if need be.  False if the range has none left.
template <int RB>
NVFP4_DEVINL bool find_tile(const Call &c, int64_t end, Item *it, int64_t *item_begin, int64_t *u)
{
    while (*u < end) {
        if (*u >= *item_begin + it->units) {
            *item_begin += it->units;
            next_item<RB, kTile>(c, it);
        }
        *u = max(*u, *item_begin + c.item_cost);
        if (*u < end)
            return true;
    }
    return false;
}

// Tiles of the item from place u on that are the CTA's.
NVFP4_DEVINL int tiles_from(const Range &range, const Item &it, int64_t item_begin, int64_t u)
{
    return (int)(min(item_begin + it.units, range.end) - u);
}

// The CTA's segments: f(number of tiles, index of the first among the CTA's) until it returns false.
template <int RB, class F>
NVFP4_DEVINL void for_segments(const Call &c, const Range &range, Item it, int64_t item_begin, F &&f)
{
    uint32_t tile = 0;
    for (int64_t u = range.begin; find_tile<RB>(c, range.end, &it, &item_begin, &u);) {
        const int n = tiles_from(range, it, item_begin, u);
        if (!f(n, tile))
            return;
        tile += n;
        u += n;
    }
}

// The tiles of a CTA's range, one by one.
template <int RB>
struct TileCursor {
    Item it;
    int64_t item_begin, u, end;

    // to the first tile from u on
    NVFP4_DEVINL void settle(const Call &c) { find_tile<RB>(c, end, &it, &item_begin, &u); }
    NVFP4_DEVINL int key0(const Call &c) const { return (it.tile0 + (int)(u - item_begin - c.item_cost)) * kTile; }
};

// ---------------------------------------------------------------------------
// Load warp
// ---------------------------------------------------------------------------

// A tile is cut into runs that lie in one page each (16 keys at least); lane i
// copies run i, a whole page in one piece.  Runs that no row sees, and pages that are not there, are not
// copied.
template <int FMT, int D, bool SPLIT>
NVFP4_DEVINL bool load_role(const Call &c, const Range &range, const Item &first, int64_t item_begin, Shared *sh,
                            uint32_t smem, int is_v, int lane)
{
    using C = Cfg<FMT, D, SPLIT>;
    using R = kv::Row<FMT, D>;
    const uint32_t n = is_v ? C::kRawVs : C::kRawKs;  // buffers
    const int shift = c.pool.page_shift, run = min(1 << shift, kTile), runs = kTile / run;
    TileCursor<C::kRows> cur{first, item_begin, range.begin, range.end};
    const uint32_t tiles = sh->tiles;
    // Page numbers of 32 runs of the item at a time, and of the 32 behind them:
    // a table read per tile took longer than everything else the warp does.
    const auto look_up = [&](uint32_t key) {  // (unsigned: 63 runs beyond a tile may pass 2^31)
        const bool sees = key < (uint32_t)cur.it.hi && (int)key + run > cur.it.lo;
        return sees ? c.table[(int64_t)cur.it.b * c.table_width + (key >> shift)] : -1;
    };
    int pages = 0, pages_behind = 0, used = 32;  // runs of `pages` that are behind us
    int64_t item_of_pages = -1;
    int all_lo = 0, all_hi = 0;
    bool ok = true;
    uint32_t tile = 0;
#pragma unroll 1
    for (; tile < tiles; ++tile) {
        cur.settle(c);
        const int key0 = cur.key0(c), key = key0 + lane * run, head = cur.it.head;
        if (item_of_pages != cur.item_begin) {
            item_of_pages = cur.item_begin;
            common_keys(c, cur.it, &all_lo, &all_hi);
            pages = look_up(key0 + lane * run);
            pages_behind = look_up((uint32_t)key0 + (32 + lane) * run);
            used = 0;
        } else if (used == 32) {
            pages = pages_behind;
            pages_behind = look_up((uint32_t)key0 + (32 + lane) * run);
            used = 0;
        }
        const int page = __shfl_sync(0xFFFFFFFFu, pages, (used + lane) & 31);
        used += runs;
        const bool want = lane < runs && key < cur.it.hi && key + run > cur.it.lo;
        const bool there = want && page >= 0 && page < c.pool.n_pages;
        if (want && !there)
            kv::report_index(c.pool.status, kStatusKvAttention);
        const uint32_t missing = __ballot_sync(0xFFFFFFFFu, want && !there);
        const uint32_t copied = __popc(__ballot_sync(0xFFFFFFFFu, there));
        RawInfo info{key0, cur.it.lo, cur.it.hi, all_lo, all_hi, 0};
#pragma unroll
        for (int g = 0; g < kTile / 16; ++g)
            info.present |= (missing >> (g * 16 / run) & 1 ? 0u : 1u) << g;
        const uint8_t *const k = kv::block_ptr(c.pool, there ? page : 0, head, 0);
        const uint8_t *const v = k + c.pool.block_bytes;
        const int at = key & ((1 << shift) - 1);
        const uint32_t scales = R::kCode << shift, exps = (R::kCode + R::kScale) << shift;
        ++cur.u;
        const uint32_t slot = tile % n, round = tile / n;
        ok = round == 0 || tc::mbar_wait(&sh->raw_empty[is_v][slot], (round - 1) & 1);
        if (!(ok = __all_sync(0xFFFFFFFFu, ok)))
            break;
        if (lane == 0) {
            sh->raw[is_v][slot] = info;
            tc::mbar_arrive_expect_tx(&sh->raw_full[is_v][slot], copied * run * (R::kBytes + (is_v ? 0 : 1)));
        }
        __syncwarp();
        if (there) {
            const uint8_t *const from = is_v ? v : k;
            const uint32_t full = tc::smem_addr(&sh->raw_full[is_v][slot]);
            const uint32_t dst = smem + (is_v ? C::kRawVAt + slot * C::kRawVBytes : C::kRawKAt + slot * C::kRawKBytes);
            const uint32_t to = dst + lane * run * R::kBytes;
            if (run == 1 << shift) {  // a whole page: its codes, scales and exponents are one piece
                tc::bulk_load_a(to, from, run * R::kBytes, full);
            } else {
                tc::bulk_load_a(to, from + at * R::kCode, run * R::kCode, full);
                if (R::kScale)
                    tc::bulk_load_a(to + run * R::kCode, from + scales + at * R::kScale, run * R::kScale, full);
                tc::bulk_load_a(to + run * (R::kCode + R::kScale), from + exps + at, run, full);
            }
            if (!is_v)
                tc::bulk_load_a(dst + C::kRawRows + lane * run, v + exps + at, run, full);
        }
    }
    // nothing is in flight when the warp leaves
    for (uint32_t t = tile > n ? tile - n : 0; t < tile; ++t)
        ok = tc::mbar_wait(&sh->raw_full[is_v][t % n], (t / n) & 1) && ok;
    return ok;
}

// ---------------------------------------------------------------------------
// Conversion warps
// ---------------------------------------------------------------------------

// f16x2 of 2^x, zero below 2^-24.
NVFP4_DEVINL uint32_t pow2_f16x2(int x)
{
    const float f = x < -40 ? 0.f : __uint_as_float((uint32_t)(127 + x) << 23);
    return f32x2_to_f16x2(f, f);
}

// Exponent bytes, four to a lane: 0 is a row that nobody sees, 255 one that is not a number.
//
// The warp's largest of rows that hold numbers; 0 or less if there is none.
NVFP4_DEVINL int largest_exp(uint32_t four)
{
    const uint32_t a = (four & 0x00FF00FFu) + 0x00010001u, b = (four >> 8 & 0x00FF00FFu) + 0x00010001u;  // e + 1 mod 256
    const uint32_t m = __vmaxu2(a & 0x00FF00FFu, b & 0x00FF00FFu);
    return (int)__reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16)) - 1;
}
NVFP4_DEVINL int unit_of(int largest) { return largest <= 27 ? 127 : largest; }  // (27: all zero)

// A lane's smallest of rows that hold numbers other than zero (e = 27 is the
// smallest that the append writes: such a row counts as zero); from 255 on: there is none.
NVFP4_DEVINL int smallest_of(uint32_t four)
{
    const uint32_t a = (four & 0x00FF00FFu) + 0x00E400E4u, b = (four >> 8 & 0x00FF00FFu) + 0x00E400E4u;  // e - 28 mod 256
    const uint32_t m = __vminu2(a & 0x00FF00FFu, b & 0x00FF00FFu);
    return (int)min(m & 0xFFFFu, m >> 16) + 28;
}

// Bytes j of a word for keys first + j that lie in [lo, hi), all ones.
NVFP4_DEVINL uint32_t range_bytes(int first, int lo, int hi)
{
    uint32_t m = 0xFFFFFFFFu;
    if (first < lo)
        m = first + 4 <= lo ? 0u : m << (8 * (lo - first));
    if (first + 4 > hi)
        m &= first >= hi ? 0u : 0xFFFFFFFFu >> (8 * (first + 4 - hi));
    return m;
}

// Exponent byte of V's unit in a tile whose rows see different keys; its largest
// exponent is `top`.  all: bytes of the keys that every row sees.
template <int ABOVE>
NVFP4_DEVINL int mixed_unit(uint32_t four, uint32_t all, int top, bool *bad)
{
    int from = largest_exp(four & all);
    if (from <= 27)  // a row may see any one of the others alone
        from = min(top, (int)__reduce_min_sync(0xFFFFFFFFu, (uint32_t)smallest_of(four)));
    const int unit = max(from, top - ABOVE);
    *bad |= unit > from + kUnseen;
    return unit;
}

// Whether a tile's rows lie too far from its units; bad: so says mixed_unit.
NVFP4_DEVINL bool is_far(uint32_t k4, uint32_t v4, int k_unit, int v_unit, bool bad)
{
    bad |= smallest_of(k4) < k_unit - kBelow || smallest_of(v4) < v_unit - kBelow || (uint32_t)(v_unit - 127 + kNear) > 2u * kNear;
    return __any_sync(0xFFFFFFFFu, bad);
}

// A thread converts, in each of its kRowsMine rows of a tile of K or V, one
// 16-byte chunk of codes of every 64-element column block; two rows (from its
// i0-th on) a call, which keeps the loop short.  Neighbouring lanes take the chunks of a block, then the next row; every
// other group of rows begins with the other block, so that both the reads (rows
// of codes) and the writes (swizzled rows of f16) of 8 lanes lie on different
// banks.  unit[i]: f16x2 factor of row i; keep[i]: all ones, or zero for a row
// that is written as zeros whatever lies in the buffer.
template <int FMT, int D, bool SPLIT>
NVFP4_DEVINL void convert(uint32_t raw, int run, uint32_t operand, int tid, int i0, const uint32_t (&unit)[2], const uint32_t (&keep)[2])
{
    using C = Cfg<FMT, D, SPLIT>;
    using R = kv::Row<FMT, D>;
    constexpr int per = C::kPerBlock, rows = 2, kOut = 8 / per;  // 16-byte chunks of f16 from one of codes
    const int row0 = tid / per + i0 * C::kRowStep, place = tid % per;
    const int flip = D == 64 ? 0 : per == 4 ? row0 & 1 : row0 >> 1 & 1;
    uint32_t swizzled[kOut];
#pragma unroll
    for (int h = 0; h < kOut; ++h)
        swizzled[h] = operand + row0 * 128 + (((place * kOut + h) ^ (row0 & 7)) << 4);
#pragma unroll 1
    for (int b = 0; b < D / 64; ++b) {
        const int block = b ^ flip;
        uint4 code[rows];
        uint32_t two[rows];
#pragma unroll
        for (int i = 0; i < rows; ++i) {
            const int row = row0 + i * C::kRowStep, in_run = row & (run - 1);
            const uint32_t from = raw + (row - in_run) * R::kBytes;  // the row's run
            code[i] = tc::lds128(from + in_run * R::kCode + (block * per + place) * 16);
            if constexpr (FMT == NVFP4_KV_NVFP4)
                two[i] = tc::lds16(from + run * R::kCode + in_run * R::kScale + (block * per + place) * 2);
        }
#pragma unroll
        for (int i = 0; i < rows; ++i) {
            const uint32_t w[4] = {code[i].x & keep[i], code[i].y & keep[i], code[i].z & keep[i], code[i].w & keep[i]};
            const uint32_t to = block * (128 * 128) + i * C::kRowStep * 128;
            if constexpr (FMT == NVFP4_KV_E4M3) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
                            : "=r"(o[2 * j]), "=r"(o[2 * j + 1])
                            : "r"(w[2 * h + j]));
                    tc::sts128(swizzled[h] + to, make_uint4(sk::f16x2_mul(o[0], unit[i]), sk::f16x2_mul(o[1], unit[i]),
                                                        sk::f16x2_mul(o[2], unit[i]), sk::f16x2_mul(o[3], unit[i])));
                }
            } else {
                const uint32_t sc = kv::without_nan(two[i] & keep[i]);
                const uint32_t s[2] = {sk::f16x2_mul(e4m3x2_to_f16x2((uint16_t)((sc & 0xFFu) * 0x101u)), unit[i]),
                                       sk::f16x2_mul(e4m3x2_to_f16x2((uint16_t)((sc >> 8) * 0x101u)), unit[i])};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t o[4];
                    sk::e2m1x8_to_f16x2(w[h], o);
                    const uint32_t m = s[h / 2];
                    tc::sts128(swizzled[h] + to, make_uint4(sk::f16x2_mul(o[0], m), sk::f16x2_mul(o[1], m),
                                                        sk::f16x2_mul(o[2], m), sk::f16x2_mul(o[3], m)));
                }
            }
        }
    }
}

// Takes the codes that are not a number out of what the thread converts of a
// tile of V (see clear_nan_codes in attention_decode.cuh; block scales: convert).
template <int FMT, int D, bool SPLIT>
NVFP4_DEVINL void clear_nan_codes(uint32_t raw, int run, int tid)
{
    using C = Cfg<FMT, D, SPLIT>;
    using R = kv::Row<FMT, D>;
    constexpr int per = C::kPerBlock;
    asm volatile("" : "+r"(tid), "+r"(run), "+r"(raw));  // nothing of this is kept ready in the loop over the tiles
#pragma unroll 1
    for (int i = 0; i < C::kRowsMine; ++i) {
        const int row = tid / per + i * C::kRowStep, in_run = row & (run - 1);
#pragma unroll 1
        for (int b = 0; b < D / 64; ++b) {
            const uint32_t at = raw + (row - in_run) * R::kBytes + in_run * R::kCode + (b * per + tid % per) * 16;
            const uint4 w = tc::lds128(at);
            tc::sts128(at, make_uint4(kv::without_nan(w.x), kv::without_nan(w.y), kv::without_nan(w.z), kv::without_nan(w.w)));
        }
    }
}

// Four warps have K's tiles and four V's, so that one's waits and fences overlap
// the other's arithmetic (the same eight warps doing K, then V, of each tile took
// 2400 clocks a tile).
template <int FMT, int D, bool SPLIT>
NVFP4_DEVINL bool convert_role(uint32_t tiles, int run, Shared *sh, uint32_t smem, int is_v, int tid)
{
    using C = Cfg<FMT, D, SPLIT>;
    using R = kv::Row<FMT, D>;
    constexpr int per = C::kPerBlock, mine = C::kRowsMine;
    const int lane = tid % 32;
    const uint32_t slots = is_v ? C::kRawVs : C::kRawKs;
    uint64_t *const full = is_v ? sh->v_full : sh->k_full, *const empty = is_v ? sh->v_empty : sh->k_empty;
    const uint32_t operand = smem + (is_v ? C::kVAt : C::kKAt);
    for (uint32_t tile = 0; tile < tiles; ++tile) {
        const uint32_t st = tile % kStages, ph = (tile / kStages) & 1, slot = tile % slots;
        const uint32_t raw = smem + (is_v ? C::kRawVAt + slot * C::kRawVBytes : C::kRawKAt + slot * C::kRawKBytes);
        bool ok = tc::mbar_wait(&sh->raw_full[is_v][slot], (tile / slots) & 1);
        ok = ok && (tile < kStages || tc::mbar_wait(&empty[st], ph ^ 1));
        if (!__all_sync(0xFFFFFFFFu, ok))
            return false;
        // exponents of rows 4 lane .. 4 lane + 3, a byte each; 0: no row that anyone sees
        const RawInfo info = sh->raw[is_v][slot];
        const int in_run = 4 * lane & (run - 1);
        uint32_t own = tc::lds32(raw + (4 * lane - in_run) * R::kBytes + run * (R::kCode + R::kScale) + in_run);
        uint32_t other = is_v ? own : tc::lds32(raw + C::kRawRows + 4 * lane);
        const int first = info.key0 + 4 * lane;
        const uint32_t keep = info.present >> (lane / 4) & 1 ? range_bytes(first, info.lo, info.hi) : 0u;
        own &= keep;
        other &= keep;
        const bool mixed = info.mixed();
        int v_unit = unit_of(largest_exp(other));
        bool bad = false;
        if (mixed) {
            if (FMT == NVFP4_KV_E4M3 && is_v)
                clear_nan_codes<FMT, D, SPLIT>(raw, run, tid);
            v_unit = mixed_unit<C::kAbove>(other, range_bytes(first, info.all_lo, info.all_hi), v_unit, &bad);
        }
        const int top = is_v ? v_unit : unit_of(largest_exp(own));
        const bool far = !is_v && is_far(own, other, top, v_unit, bad);
#pragma unroll 1
        for (int i0 = 0; i0 < mine; i0 += 2) {
            uint32_t unit[2], rows[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = tid / per + (i0 + i) * C::kRowStep, sh8 = 8 * (row & 3);
                const uint32_t a = __shfl_sync(0xFFFFFFFFu, own, row >> 2) >> sh8 & 0xFFu;
                const uint32_t b = __shfl_sync(0xFFFFFFFFu, other, row >> 2) >> sh8 & 0xFFu;
                // a row that is not a number makes its scores NaN, whichever of K and V it is, and V's are zero
                unit[i] = a == kv::kNanRow || b == kv::kNanRow ? (is_v ? 0u : 0x7FFF7FFFu) : pow2_f16x2((int)a - top);
                rows[i] = a != 0 ? 0xFFFFFFFFu : 0u;
            }
            convert<FMT, D, SPLIT>(raw, run, operand + st * C::kOperand, tid, i0, unit, rows);
        }
        if (!is_v && tid == 0)
            sh->info[tile % kInfos] = {kv::exp2_byte(top), (float)(v_unit - 127), far ? 0u : info.present, 0};
        if (far && tid == 0)
            sh->far_tile = tile + 1;
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tc::mbar_arrive(&full[st]);
            tc::mbar_arrive(&sh->raw_empty[is_v][slot]);
        }
    }
    return true;
}

// ---------------------------------------------------------------------------
// MMA warps
// ---------------------------------------------------------------------------

template <int FMT, int D, bool SPLIT>
NVFP4_DEVINL bool mma_role(const Call &c, const Range &range, const Item &first, int64_t item_begin, Shared *sh,
                           uint32_t smem, uint32_t tmem, int group)
{
    using C = Cfg<FMT, D, SPLIT>;
    constexpr uint32_t score_idesc = tc::idesc_f16kind(128, kTile / 2, 0);
    constexpr uint32_t out_idesc = tc::idesc_f16kind(128, D, 0) | 1u << 16;  // B transposed
    const uint32_t scores = tmem + C::kScoreCols + group * kTile, out = tmem + C::kOutCols + group * D;
    const uint32_t q = smem + C::kQAt + (SPLIT ? 0 : group) * C::kOperand;
    bool ok = true;
    uint32_t segments = 0, mine = 0;  // of this group so far: segments, and tiles whose scores were begun
    // scores of half h of the group's tile number `t`, which is the CTA's number `tile`
    const auto score = [&](uint32_t t, uint32_t tile, int h) {
        const uint32_t st = tile % kStages, ph = (tile / kStages) & 1;
        // (the half's weights of the tile before lie where its scores go)
        ok = ok && (h == 1 || tc::mbar_wait(&sh->k_full[st], ph)) &&
             (t == 0 || tc::mbar_wait(&sh->pv_done[group][h], (t - 1) & 1));
        if (!ok)
            return;
        tc::fence_after_sync();
        const uint32_t k = smem + C::kKAt + st * C::kOperand + h * (kTile / 2) * 128;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            const uint32_t at = (d / 4) * (128 * 128) + (d % 4) * 32;
            const uint64_t base = 1ull << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
            tc::mma_bf16_ss(scores + h * (kTile / 2), base | ((q + at) & 0x3FFFFu) >> 4, base | ((k + at) & 0x3FFFFu) >> 4,
                            score_idesc, d > 0);
        }
        tc::mma_commit(&sh->s_full[group][h]);
        if (h == 1)
            tc::mma_commit(&sh->k_empty[st]);
    };
    for_segments<C::kRows>(c, range, first, item_begin, [&](int n, uint32_t tile) {
        if (!has_tile<SPLIT>(group, tile, n))
            return true;
        ok = tc::mbar_wait(&sh->q_ready[group], segments++ & 1);
        constexpr uint32_t step = SPLIT ? 2 : 1;
        const uint32_t end = tile + n;
        tile += SPLIT ? (tile ^ group) & 1 : 0;
        score(mine, tile, 0);
        bool begun = false;
#pragma unroll 1
        for (; tile < end && ok; tile += step, ++mine) {
            const uint32_t st = tile % kStages, ph = (tile / kStages) & 1;
            const uint32_t v = smem + C::kVAt + st * C::kOperand;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                // the next scores are made while the softmax is at these; those of the
                // next tile wait behind this product if its keys are not converted yet
                const bool more = tile + step < end;
                const uint32_t next = tile + step;
                bool made = true;
                if (h == 0)
                    score(mine, tile, 1);
                else if (more && (made = tc::mbar_try_wait(&sh->k_full[next % kStages], (next / kStages) & 1)))
                    score(mine + 1, next, 0);
                ok = ok && (h == 1 || tc::mbar_wait(&sh->v_full[st], ph)) && tc::mbar_wait(&sh->p_ready[group][h], mine & 1);
                if (!ok)
                    break;
                tc::fence_after_sync();
#pragma unroll
                for (int j = 0; j < kTile / 32; ++j)
                    tc::mma_f16_ts(out, scores + h * (kTile / 2) + 8 * j, desc_transposed(v + (h * (kTile / 32) + j) * 2048),
                                   out_idesc, begun || j > 0);
                tc::mma_commit(&sh->pv_done[group][h]);
                if (h == 1)
                    tc::mma_commit(&sh->v_empty[st]);
                begun = true;
                if (!made)
                    score(mine + 1, next, 0);
            }
        }
        return ok;
    });
    // nothing of this thread's is in flight when it leaves
    tc::mma_commit(&sh->drain[group]);
    return tc::mbar_wait(&sh->drain[group], 0) && ok;
}

// ---------------------------------------------------------------------------
// Softmax warps
// ---------------------------------------------------------------------------

// Bits j of a word for keys first + j that lie in [lo, hi).
NVFP4_DEVINL uint32_t range_bits(int first, int lo, int hi)
{
    const int a = max(lo - first, 0), b = min(hi - first, 32);
    return a >= b ? 0u : (0xFFFFFFFFu << a) & (0xFFFFFFFFu >> (32 - b));
}

// Keys first .. first + 31 that a row sees.
NVFP4_DEVINL uint32_t seen_bits(int first, int lo, int hi, bool tree, uint64_t word, int past)
{
    uint32_t m = range_bits(first, lo, hi);
    if (tree) {
        const int o = first - past;  // of key `first` among the new tokens
        uint32_t t;
        if (o >= 64)
            t = 0;
        else if (o >= 0)
            t = (uint32_t)(word >> o);
        else
            t = o <= -32 ? 0xFFFFFFFFu : (uint32_t)(word << -o) | ((1u << -o) - 1);
        m &= t;
    }
    return m;
}

// The next segment from place g->u on.
template <int RB>
NVFP4_DEVINL void find_segment(const Call &c, const Range &range, Segment *g)
{
    Item it = g->it;
    int64_t item_begin = g->item_begin, u = g->u;
    const bool any = find_tile<RB>(c, range.end, &it, &item_begin, &u);
    g->it = it;
    g->item_begin = item_begin;
    g->u = u;
    g->n = any ? tiles_from(range, it, item_begin, u) : 0;
    g->tile0 = any ? it.tile0 + (int)(u - item_begin - c.item_cost) : 0;
}

// f32 of 8 elements of a row (from element 8 i on): its codes, times its block scale.
template <int FMT, int D>
NVFP4_DEVINL void eight_elements(const uint8_t *blk, int shift, int at, int i, float (&x)[8])
{
    using R = kv::Row<FMT, D>;
    uint32_t h[4];
    float scale = 1.f;
    if constexpr (FMT == NVFP4_KV_E4M3) {
        const uint2 w = *reinterpret_cast<const uint2 *>(blk + at * R::kCode + i * 8);
        h[0] = e4m3x2_to_f16x2((uint16_t)w.x), h[1] = e4m3x2_to_f16x2((uint16_t)(w.x >> 16));
        h[2] = e4m3x2_to_f16x2((uint16_t)w.y), h[3] = e4m3x2_to_f16x2((uint16_t)(w.y >> 16));
    } else {
        sk::e2m1x8_to_f16x2(*reinterpret_cast<const uint32_t *>(blk + at * R::kCode + i * 4), h);
        scale = e4m3_to_f32(blk[(R::kCode << shift) + at * R::kScale + i / 2]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float lo, hi;
        asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }" : "=f"(lo), "=f"(hi) : "r"(h[j]));
        x[2 * j] = lo * scale;
        x[2 * j + 1] = hi * scale;
    }
}

// The far tiles of a segment, which the tensor cores were told are not there: a
// thread computes its row's scores and weights in fp32, with each key's own
// exponents, and adds them to the row's accumulators, reference and sum.  About 0.2 ms
// a tile (of 128 or 256 rows): its aims are to be right and short.
template <int FMT, int D, bool SPLIT>
NVFP4_DEVINL void far_tiles(const Call &c, const Segment &g, uint32_t q_at, uint32_t out, int group, int r, int lo, int hi,
                            bool tree, uint64_t word, float factor, float *top, float *sum)
{
    using C = Cfg<FMT, D, SPLIT>;
    using R = kv::Row<FMT, D>;
    const int lane = r % 32, shift = c.pool.page_shift, mask = (1 << shift) - 1, past = g.it.seq.past;
    const int32_t *const table = c.table + (int64_t)g.it.b * c.table_width;
    const auto block = [&](int key) -> const uint8_t * {  // K's of the key's page, or null
        const int page = key >= g.it.lo && key < g.it.hi ? table[key >> shift] : -1;
        return page >= 0 && page < c.pool.n_pages ? kv::block_ptr(c.pool, page, g.it.head, 0) : nullptr;
    };
    int all_lo, all_hi;
    common_keys(c, g.it, &all_lo, &all_hi);
#pragma unroll 1
    for (int i = SPLIT ? (int)((g.index ^ group) & 1) : 0; i < g.n; i += SPLIT ? 2 : 1) {
        const int key0 = (g.tile0 + i) * kTile;
        {
            // the conversion's rules again
            uint32_t k4 = 0, v4 = 0;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const int key = key0 + 4 * lane + j;
                if (const uint8_t *blk = block(key)) {
                    const int at = ((R::kCode + R::kScale) << shift) + (key & mask);
                    k4 |= (uint32_t)blk[at] << 8 * j;
                    v4 |= (uint32_t)blk[at + c.pool.block_bytes] << 8 * j;
                }
            }
            bool bad = false;
            int v_unit = unit_of(largest_exp(v4));
            if (max(key0, g.it.lo) < all_lo || min(key0 + kTile, g.it.hi) > all_hi)
                v_unit = mixed_unit<C::kAbove>(v4, range_bytes(key0 + 4 * lane, all_lo, all_hi), v_unit, &bad);
            if (!is_far(k4, v4, unit_of(largest_exp(k4)), v_unit, bad))
                continue;
        }
        float next = *top, base = 0.f, shrink = 1.f, largest = -INFINITY, l = 0.f;
        float z_of[kTile];  // (in local memory)
        // first the largest z = score + V's exponent, then 32 elements of the output at a time
#pragma unroll 1
        for (int pass = -1; pass < D / 32; ++pass) {
            float acc[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                acc[j] = 0.f;
#pragma unroll 1
            for (int key = key0; key < key0 + kTile; ++key) {
                const uint8_t *const blk = block(key);
                if (!blk)
                    continue;
                const int at = key & mask, e_at = ((R::kCode + R::kScale) << shift) + at;
                const uint32_t ve = blk[e_at + c.pool.block_bytes];
                const float kv = __uint_as_float(0x4B000000u | ve) - 8388735.f;
                if (pass < 0) {
                    bool see = key >= lo && key < hi;
                    if (tree && key >= past)
                        see &= key - past < 64 && (word >> ((key - past) & 63) & 1);
                    float score = 0.f;
#pragma unroll 1
                    for (int d = 0; d < D / 8; ++d) {
                        float x[8];
                        eight_elements<FMT, D>(blk, shift, at, d, x);
                        const uint4 q = tc::lds128(operand_chunk(q_at, r, d));
                        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float a, b;
                            asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }" : "=f"(a), "=f"(b) : "r"(w[j]));
                            score = fmaf(a, x[2 * j], score);
                            score = fmaf(b, x[2 * j + 1], score);
                        }
                    }
                    score = score * factor * kv::exp2_byte(blk[e_at]);
                    const float z = !see ? -INFINITY : ve == kv::kNanRow ? NAN : score + kv;
                    z_of[key - key0] = z;
                    largest = fmaxf(largest, z);
                } else {
                    const float z = z_of[key - key0], w = ex2(z - base);
                    if (pass == 0)
                        l += ex2_subnormal(z - (base + kv + 32.f));  // in units of kSumUnit
                    if (w != 0.f) {  // (true for a NaN; a zero must not meet what an unseen row holds)
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            float x[8];
                            eight_elements<FMT, D>(blk + c.pool.block_bytes, shift, at, 4 * pass + d, x);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                acc[8 * d + j] = fmaf(w, x[j], acc[8 * d + j]);
                        }
                    }
                }
            }
            if (pass < 0) {
                next = fmaxf(*top, largest - kHeadroom);
                base = next == -INFINITY ? 0.f : next;
                shrink = *top == next ? 1.f : ex2(*top - next);
                continue;
            }
            uint32_t x[32];
            __syncwarp();
            tc::tmem_ld_32x32b_x32(out + 32 * pass, x);
            tc::tmem_ld_wait();
            settle(x);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = __float_as_uint(fmaf(__uint_as_float(x[j]), shrink, acc[j]));
            tc::tmem_st_32x32b_x32(out + 32 * pass, x);
        }
        if (*top != next)
            *sum = times_pow2(*sum, *top - next);
        *sum += l;
        *top = next;
    }
    tc::tmem_st_wait();
}
static_assert(kSumUnit == 0x1p-32f, "far_tiles");

// The segment lies in shared memory, not in registers: the loop over the tiles
// needs those for the scores.
template <int FMT, int D, bool SPLIT>
NVFP4_DEVINL bool softmax_role(const Call &c, const Range &range, Shared *sh, uint32_t smem, uint32_t tmem,
                               uint8_t *workspace, int tid)
{
    using C = Cfg<FMT, D, SPLIT>;
    constexpr int kBar = 1, kAll = 32 * kSoftmaxWarps;
    const int group = tid / 128, r = tid % 128;       // row of the row tile, and lane of tensor memory
    const uint32_t lanes = (uint32_t)(r & ~31) << 16;
    const uint32_t scores = tmem + C::kScoreCols + group * kTile + lanes;
    const uint32_t out = tmem + C::kOutCols + group * D + lanes;
    const Segment &g = sh->seg;
    float2 (*const stats)[kRowTile] = reinterpret_cast<float2 (*)[kRowTile]>(reinterpret_cast<uint8_t *>(sh) - C::kStatsBytes);  // SPLIT: of a row, by group
    bool ok = true;
    uint32_t mine = 0;

    for (;;) {
        const int row = (SPLIT ? 0 : group * kRowTile) + r;  // row of the item
        const bool live = row < g.it.rows;
        const auto token = [&] { return (g.it.row0 + row) / c.group; };
        // rows beyond the last one: no key is masked, and none has any weight
        int lo = 0, hi = INT32_MAX;
        uint64_t word = 0;
        float top = 1e30f;
        const int past = g.it.seq.past;
        int64_t q_at_elem = 0;
        if (live) {
            const int tok = token();
            const int64_t q_row = g.it.seq.q_begin + tok;
            key_range(c, g.it.seq, tok, &lo, &hi);
            if (c.tree)
                word = c.tree[q_row];
            top = -INFINITY;
            q_at_elem = q_row * c.q_ld + (int64_t)(g.it.head * c.group + (g.it.row0 + row) - tok * c.group) * D;
        }
        // Q to f16, times a power of two that puts its largest element at 2^14 (and the scale's sign)
        float factor = 0.f;
        if (!SPLIT || group == 0) {
            const uint32_t q_at = smem + C::kQAt + (SPLIT ? 0 : group) * C::kOperand;
            const uint4 *src = reinterpret_cast<const uint4 *>(c.q + q_at_elem);
            uint32_t m2 = 0;
            if (live) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 x = src[i];
                    m2 = __vmaxu2(__vmaxu2(m2, x.x & 0x7FFF7FFFu), x.y & 0x7FFF7FFFu);
                    m2 = __vmaxu2(__vmaxu2(m2, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
                }
            }
            const int e = max((int)(max(m2 & 0xFFFFu, m2 >> 16) >> 7), 15);
            const float sign = c.scale_log2 < 0 ? -1.f : c.scale_log2 > 0 ? 1.f : 0.f;
            const float up = (e == 255 ? NAN : __uint_as_float((uint32_t)(268 - e) << 23)) * sign;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint4 x = live ? src[i] : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[j] = f32x2_to_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
                tc::sts128(operand_chunk(q_at, r, i), make_uint4(h[0], h[1], h[2], h[3]));
            }
            factor = fabsf(c.scale_log2) * __uint_as_float((uint32_t)(e - 14) << 23);
            if (SPLIT)
                stats[0][r].x = factor;
            tc::fence_proxy_async_smem();
            // a group waits once for each segment in which it has a tile
            for (int i = SPLIT ? 0 : group; i <= (SPLIT ? 1 : group); ++i) {
                if (has_tile<SPLIT>(i, g.index, g.n))
                    tc::mbar_arrive(&sh->q_ready[i]);
            }
        }
        if (SPLIT) {
            tc::named_bar_sync(kBar, kAll);
            factor = stats[0][r].x;
        }

        float sum = 0.f;
        bool begun = false;
        const int n = g.n, tile0 = g.tile0;
        const uint32_t index = g.index;
        for (int i = SPLIT ? (int)((index ^ group) & 1) : 0; i < n && ok; i += SPLIT ? 2 : 1) {
            const int key0 = (tile0 + i) * kTile;
            ok = tc::mbar_wait(&sh->s_full[group][0], mine & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok)
                break;
            const TileInfo info = sh->info[(index + i) % kInfos];
            // above zero: a masked score of -infinity stays one
            const float f = fmaxf(factor * info.k_unit, 0x1p-126f);
            const bool whole = __all_sync(0xFFFFFFFFu, key0 >= lo && key0 + kTile <= (c.tree && live ? min(hi, past) : hi) &&
                                                           info.present == 0xFFu);
            const float sum_unit = ex2(-info.v_exp) * kSumUnit;
            const uint64_t f2 = pack2(f, f);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // halves of the keys
                if (h == 1) {
                    ok = tc::mbar_wait(&sh->s_full[group][1], mine & 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok)
                        break;
                }
                tc::fence_after_sync();
                uint32_t s[2][32];
                tc::tmem_ld_32x32b_x32(scores + 64 * h, s[0]);
                tc::tmem_ld_32x32b_x32(scores + 64 * h + 32, s[1]);
                tc::tmem_ld_wait();
                settle(s[0]);
                settle(s[1]);
                bool sees = true;
                if (!whole) {
                    sees = false;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int at = 4 * h + 2 * q;
                        uint32_t see = seen_bits(key0 + 16 * at, lo, hi, c.tree && live, word, past);
                        see &= (info.present >> at & 1 ? 0x0000FFFFu : 0u) | (info.present >> at & 2 ? 0xFFFF0000u : 0u);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            s[q][j] = see >> j & 1 ? s[q][j] : 0xFF800000u;  // -infinity
                        sees |= see != 0;
                    }
                }
                float l = 0.f;
                bool over = top == -INFINITY && sees;
                // at most twice: after the move no weight is above 2^kHeadroom
#pragma unroll 1
                for (int pass = 0; pass < 2; ++pass) {
                    if (__any_sync(0xFFFFFFFFu, over)) {
                        // move the row's reference to its largest score so far, and with it what was summed up
                        float m = -INFINITY;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
#pragma unroll
                            for (int j = 0; j < 32; j += 2)
                                m = max3(m, __uint_as_float(s[q][j]), __uint_as_float(s[q][j + 1]));
                        }
                        const float next = over ? fmaxf(top, fmaf(m, f, info.v_exp) - kHeadroom) : top;
                        // (nothing has been summed before the first reference)
                        const float shrink = top == next || top == -INFINITY ? 1.f : ex2(top - next);
                        top = next;
                        sum *= shrink;
                        const bool move = __any_sync(0xFFFFFFFFu, shrink != 1.f);
                        if (move && (begun || h == 1)) {
                            // the half's before product may be under way
                            ok = ok && tc::mbar_wait(&sh->pv_done[group][h ^ 1], (h == 1 ? mine : mine - 1) & 1);
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t x[16];
                                tc::tmem_ld_32x32b_x16(out + 16 * q, x);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    asm volatile("mul.rn.f32 %0, %0, %1;" : "+r"(x[j]) : "f"(shrink));
                                tc::tmem_st_32x32b_x16(out + 16 * q, x);
                            }
                        }
                    }
                    const float add = info.v_exp - (top == -INFINITY ? 0.f : top);
                    const uint64_t add_2 = pack2(add, add);
                    uint64_t l2[2] = {0, 0};
                    uint32_t p[2][16];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 e = unpack2(fma2(
                                pack2(__uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1])), f2, add_2));
                            const float a = ex2(e.x), b = ex2(e.y);
                            l2[j & 1] = add2(l2[j & 1], pack2(a, b));
                            p[q][j] = f32x2_to_f16x2(a, b);
                        }
                        tc::tmem_st_32x32b_x16(scores + 64 * h + 16 * q, p[q]);
                    }
                    const float2 la = unpack2(l2[0]), lb = unpack2(l2[1]);
                    l = (la.x + la.y) + (lb.x + lb.y);
                    over = l > kMostWeight;
                    if (!__any_sync(0xFFFFFFFFu, over))
                        break;
                }
                sum = fmaf(l, sum_unit, sum);
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (r % 32 == 0)
                    tc::mbar_arrive(&sh->p_ready[group][h]);
            }
            begun = true;
            ++mine;
        }
        if (ok && begun)
            ok = tc::mbar_wait(&sh->pv_done[group][1], (mine - 1) & 1);
        ok = tc::bar_and(kBar, kAll, ok);
        if (!ok)
            return false;
        tc::fence_after_sync();
        if (sh->far_tile > index)
            far_tiles<FMT, D, SPLIT>(c, g, smem + C::kQAt + (SPLIT ? 0 : group) * C::kOperand, out, group, r, lo, live ? hi : 0,
                                     c.tree, word, factor, &top, &sum);

        // The row's result: with SPLIT, the two groups' joined, each group taking half of the elements.
        constexpr int kCols = SPLIT ? D / 2 : D;
        const int col0 = SPLIT ? group * kCols : 0;
        float w_other = 0.f, w_mine = 1.f;
        if (SPLIT) {
            stats[group][r] = make_float2(begun ? top : -INFINITY, begun ? sum : 0.f);
            tc::named_bar_sync(kBar, kAll);
            const float2 a = stats[0][r], b = stats[1][r];
            top = fmaxf(a.x, b.x);
            // groups without a tile have nothing in tensor memory; 0 * NaN stays NaN in the others
            const float wa = a.x == -INFINITY ? 0.f : ex2(a.x - top), wb = b.x == -INFINITY ? 0.f : ex2(b.x - top);
            sum = fmaf(wa, a.y, wb * b.y);
            if (fabsf(a.x - b.x) > -kTwoSteps)  // (far tiles' references can lie that far apart)
                sum = times_pow2(a.y, a.x - top) + times_pow2(b.y, b.x - top);
            w_mine = wa;
            w_other = wb;
        }
        const bool has0 = !SPLIT || has_tile<SPLIT>(0, g.index, g.n), has1 = SPLIT && has_tile<SPLIT>(1, g.index, g.n);
        const uint32_t out0 = SPLIT ? tmem + C::kOutCols + lanes : out, out1 = tmem + C::kOutCols + D + lanes;
        const auto result = [&](int q, float (&x)[32]) {  // elements col0 + 32 q ..
            uint32_t s[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = 0.f;
            if (has0) {
                tc::tmem_ld_32x32b_x32(out0 + col0 + 32 * q, s);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] = __uint_as_float(s[j]) * w_mine;
            }
            if (has1) {
                tc::tmem_ld_32x32b_x32(out1 + col0 + 32 * q, s);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] = fmaf(__uint_as_float(s[j]), w_other, x[j]);
            }
        };
        const auto store = [&](int q, const float (&x)[32], float l) {
            if (!live)
                return;
            const float inv = l == 0.f ? 0.f : kSumUnit / l;
            const int tok = token();
            uint16_t *dst = static_cast<uint16_t *>(c.out) + (g.it.seq.q_begin + tok) * c.out_ld +
                            (int64_t)(g.it.head * c.group + (g.it.row0 + row) - tok * c.group) * D + col0 + 32 * q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = f32x2_to_bf16x2(x[8 * j + 2 * k] * inv, x[8 * j + 2 * k + 1] * inv);
                reinterpret_cast<uint4 *>(dst)[j] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        };
        const int64_t tiles_begin = g.item_begin + c.item_cost, item_end = g.item_begin + g.it.units;
        if (tiles_begin >= range.begin && item_end <= range.end) {
            for (int q = 0; q < kCols / 32; ++q) {
                float x[32];
                result(q, x);
                store(q, x, sum);
            }
        } else {
            // partial result: [element / 4][row][4], then [row] (largest, sum)
            uint32_t *const counters = reinterpret_cast<uint32_t *>(workspace + kCounterOffset);
            float *const partials = reinterpret_cast<float *>(workspace + kPartialOffset);
            const int first_cta = range_owner(range.total, range.ctas, tiles_begin);
            const int last_cta = range_owner(range.total, range.ctas, item_end - 1);
            float *slot = partials + ((int64_t)blockIdx.x * 2 + ((int)blockIdx.x == first_cta ? 1 : 0)) * C::kSlotFloats;
            for (int q = 0; q < kCols / 32; ++q) {
                float x[32];
                result(q, x);
                if (!live)
                    continue;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    reinterpret_cast<float4 *>(slot)[(col0 / 4 + 8 * q + j) * C::kRows + row] =
                        make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            }
            if (!SPLIT || group == 0)
                reinterpret_cast<float2 *>(slot + C::kRows * D)[row] = make_float2(top, sum);
            tc::named_bar_sync(kBar, kAll);  // before the release below: it covers every thread's stores
            if (tid == 0) {
                uint32_t seen;
                asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(seen) : "l"(counters + first_cta) : "memory");
                const bool done = seen == (uint32_t)(last_cta - first_cta);
                if (done)
                    counters[first_cta] = 0;
                sh->last = done;
            }
            tc::named_bar_sync(kBar, kAll);
            if (sh->last) {
                const int count = last_cta - first_cta + 1;
                const float *const from = partials + (int64_t)first_cta * 2 * C::kSlotFloats;
                const auto slot_of = [&](int i) { return from + (int64_t)(i == 0 ? 1 : 2 * i) * C::kSlotFloats; };
                const auto stats_of = [&](int i) {
                    return __ldcg(reinterpret_cast<const float2 *>(slot_of(i) + C::kRows * D) + row);
                };
                // several contributors' loads at once: one at a time, the join ran at the latency of L2
                if (live) {
                    float m = -INFINITY, l = 0.f;
#pragma unroll 4
                    for (int i = 0; i < count; ++i)
                        m = fmaxf(m, stats_of(i).x);
#pragma unroll 4
                    for (int i = 0; i < count; ++i) {
                        const float2 ml = stats_of(i);
                        l = ml.x - m < kTwoSteps ? l + times_pow2(ml.y, ml.x - m)
                                                 : fmaf(ml.x == -INFINITY ? 0.f : ex2(ml.x - m), ml.y, l);
                    }
#pragma unroll 1
                    for (int q = 0; q < kCols / 32; ++q) {
                        float x[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            x[j] = 0.f;
#pragma unroll 2
                        for (int i = 0; i < count; ++i) {
                            const float tw = stats_of(i).x;
                            const float w = tw == -INFINITY ? 0.f : ex2(tw - m);
                            const float4 *v =
                                reinterpret_cast<const float4 *>(slot_of(i)) + (col0 / 4 + 8 * q) * C::kRows + row;
                            float4 y[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                y[j] = __ldcg(v + j * C::kRows);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                x[4 * j] = fmaf(w, y[j].x, x[4 * j]);
                                x[4 * j + 1] = fmaf(w, y[j].y, x[4 * j + 1]);
                                x[4 * j + 2] = fmaf(w, y[j].z, x[4 * j + 2]);
                                x[4 * j + 3] = fmaf(w, y[j].w, x[4 * j + 3]);
                            }
                        }
                        store(q, x, l);
                    }
                }
            }
        }
        tc::fence_before_sync();
        tc::named_bar_sync(kBar, kAll);  // both groups are done with tensor memory, Q, the statistics and the segment
        if (tid == 0) {
            Segment *w = &sh->seg;
            w->u += w->n;
            w->index += w->n;
            find_segment<C::kRows>(c, range, w);
        }
        tc::named_bar_sync(kBar, kAll);
        if (g.n == 0)
            return true;
    }
}

template <int FMT, int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(Call c, uint8_t *workspace)
{
    using C = Cfg<FMT, D, SPLIT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared *const sh = reinterpret_cast<Shared *>(smem_raw + C::kBarAt);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0);

    tc::griddep_launch_dependents();
    tc::griddep_wait();
    Range range;
    Item item;
    int64_t item_begin;
    if (!find_range<C::kRows, kTile, kThreads>(c, sh->scratch, &range, &item, &item_begin))
        return;
    if (tid == 0) {
        sh->seg.it = item;
        sh->seg.item_begin = item_begin;
        sh->seg.u = range.begin;
        sh->seg.index = 0;
        sh->far_tile = 0;
        find_segment<C::kRows>(c, range, &sh->seg);
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&sh->k_full[i], kConvertWarps / 2);
            tc::mbar_init(&sh->v_full[i], kConvertWarps / 2);
            tc::mbar_init(&sh->k_empty[i], SPLIT ? 1 : 2);
            tc::mbar_init(&sh->v_empty[i], SPLIT ? 1 : 2);
        }
        for (int g = 0; g < 2; ++g) {
            tc::mbar_init(&sh->q_ready[g], kRowTile);
            for (int h = 0; h < 2; ++h) {
                tc::mbar_init(&sh->s_full[g][h], 1);
                tc::mbar_init(&sh->p_ready[g][h], kRowTile / 32);
                tc::mbar_init(&sh->pv_done[g][h], 1);
            }
            tc::mbar_init(&sh->drain[g], 1);
        }
        for (int i = 0; i < 2 * kMostRaw; ++i) {
            tc::mbar_init(&sh->raw_full[0][0] + i, 1);
            tc::mbar_init(&sh->raw_empty[0][0] + i, kConvertWarps / 2);
        }
        tc::fence_mbar_init();
    }
    if (tid == 32) {
        uint32_t tiles = 0;
        for_segments<C::kRows>(c, range, item, item_begin, [&](int n, uint32_t) {
            tiles += n;
            return true;
        });
        sh->tiles = tiles;
    }
    if (warp == kSoftmaxWarps + kConvertWarps + 2)
        tc::tmem_alloc(&sh->tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t smem = tc::smem_addr(smem_raw), tmem = sh->tmem;

    bool ok = true;
    uint32_t code = 0;
    const uint32_t tiles = sh->tiles;  // none: the range lies in the places before an item's tiles
    if (warp < kSoftmaxWarps) {
        take_regs<kSoftmaxRegs>();
        ok = tiles == 0 || softmax_role<FMT, D, SPLIT>(c, range, sh, smem, tmem, workspace, tid);
        code = kTimeoutSoftmax;
    } else if (warp < kSoftmaxWarps + kConvertWarps) {
        give_regs<kConvertRegs>();
        const int ct = tid - 32 * kSoftmaxWarps;
        ok = convert_role<FMT, D, SPLIT>(tiles, min(1 << c.pool.page_shift, kTile), sh, smem, ct / kConvertThreads,
                                         ct % kConvertThreads);
        code = kTimeoutConvert;
    } else {
        give_regs<kMmaRegs>();
        if (warp < kSoftmaxWarps + kConvertWarps + 2) {
            if (elect_one()) {
                ok = mma_role<FMT, D, SPLIT>(c, range, item, item_begin, sh, smem, tmem,
                                             warp - kSoftmaxWarps - kConvertWarps);
                code = kTimeoutMma;
            }
            __syncwarp();
        } else {
            ok = load_role<FMT, D, SPLIT>(c, range, item, item_begin, sh, smem, warp - (kSoftmaxWarps + kConvertWarps + 2),
                                          tid % 32);
            code = kTimeoutLoad;
        }
    }
    if (!ok)
        kv::report_timeout(c.pool.status, code);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kSoftmaxWarps + kConvertWarps + 2)
        tc::tmem_dealloc(tmem, 512);
}

template <int FMT, int D, bool SPLIT>
cudaError_t launch(const Call &c, uint8_t *workspace, int num_sms, cudaStream_t stream)
{
    using C = Cfg<FMT, D, SPLIT>;
    static std::once_flag once[kMaxDevices];
    static cudaError_t results[kMaxDevices];
    const auto kernel = chunk_kernel<FMT, D, SPLIT>;
    Call call = c;
    call.item_cost = kItemCost;
    const cudaError_t e = once_per_device(once, results, [kernel] {
        cudaFuncAttributes attr;
        const cudaError_t got = cudaFuncGetAttributes(&attr, kernel);
        if (got != cudaSuccess)
            return got;
        if (attr.numRegs != kLaunchRegs)  // the roles share out what the launch gives: never launch with less
            return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess)
        return e;
    return launch_dependent(kernel, dim3(num_sms < kMaxChunkCtas ? num_sms : kMaxChunkCtas), kThreads, C::kSmem, stream,
                            call, workspace);
}

template <int FMT>
cudaError_t launch_format(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if ((int64_t)c.max_q_len * c.group <= kRowTile)
        return head_dim == 64 ? launch<FMT, 64, true>(c, ws, num_sms, stream) : launch<FMT, 128, true>(c, ws, num_sms, stream);
    return head_dim == 64 ? launch<FMT, 64, false>(c, ws, num_sms, stream) : launch<FMT, 128, false>(c, ws, num_sms, stream);
}

}  // namespace chunk
}  // namespace attn
}  // namespace nvfp4
