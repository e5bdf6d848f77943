// prompt_attention.cu -- attention of packed whole prompts over their own K and V in
// bf16 (nvfp4_prompt_attention; include/nvfp4.h has the definition), on tcgen05.
//
// The two products S = Q K^T and O = P V bound it: 4 D flop for every pair of a row and a
// key that it sees, while K and V are read once per 256 rows, mostly from L2.  One persistent
// CTA per SM works on items: 2 row tiles of one sequence and KV head, and all their keys.
// A row tile is up to 128 rows: the query heads of the KV head side by side, for as many
// consecutive tokens as fit, so that grouped heads share K and V and short sequences fill tiles.
// Two row tiles are in flight so that the tensor pipe works on one while the other is in
// its softmax.  Warps by role:
//
//   warps 0-3, 4-7  softmax of row tile 0 and 1, a row to a thread: scores come from tensor
//                   memory, the weights P go back there in bf16 as the A operand of the second product
//                   (heads of 128: over the scores).  A row's reference (2^27 times its largest weight, as far as it is known)
//                   moves only where that has grown by 2^8, so that the sums so far are hardly ever multiplied.
//   warp 8          finds the items and loads Q, K and V by TMA.
//   warp 9          MMA issue of both row tiles.
//   warps 12-15     look through V tiles in which rows see different keys: an infinity or a NaN
//                   there would reach every row through 0 * inf, so it is taken out of the tile, and
//                   added at the end to the rows that do see it; and write the output rows, beside the next item's softmax.
//
// Items are taken heaviest first (the last tokens of the sequences, then those before them; of 32 sequences at a time), CTA c of P taking
// the c-th of every P, in alternating directions: for one long causal prompt every CTA then has the same
// number of keys to within a tile.  The lengths are on the device, so each CTA finds its items itself.
//
// Measured on one GB300, calls among others: 16384 tokens (40 and 8 heads of 128, causal, 2.75 TFLOP) 1.85 ms, 1.49 PFLOP/s,
// 0.76 of the measured bf16 rate (1.70 ms alone, before the power limit tells); 24 packed prompts of 19 to 2500 tokens (32 and 8
// heads) 143 us, 0.53 of it; 8191 tokens in a window of 1024 (16 and 4 heads of 64) 55 us, 5 images of 577 to 2305 tokens (16
// heads of 64) 61 us.  The weights' rounding to bf16, V's type and so the MMA's, is most of the outputs' error: 0.0008 to 0.0015 of
// their norm in fp32, 0.0018 to 0.0023 in bf16 (exact weights: 0.0016).  Two bf16 numbers a weight would double the second product.
// For a key tile of 256 rows and heads of 128 the MMAs take 2048 clocks and the whole 2800: after each S the
// MMA thread stands still until the pipe has come to it, and some 130 clocks longer before the next product begins.  With
// heads of 64 the MMAs would take 1300 and the exponentials 1024; 2300 go by: the softmax warps, two to a scheduler, issue in
// half of the clocks and wait for their own results in most others.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attention_ops.cuh"
#include "kernels.h"
#include "kv_layout.cuh"
#include "skinny.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace prompt {

using namespace attn;

constexpr int kMaxGroup = 128;  // query heads of a KV head
constexpr int kTileShift = 7, kTile = 1 << kTileShift;  // keys of a tile, rows of a row tile
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kAllocWarp = 10, kHelperWarp = 12;
// Registers of a thread by role: what the launch gives every thread, shared out anew.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 184, kOtherRegs = 72;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= kThreads * kLaunchRegs,
              "setmaxnreg would wait for registers that nobody gives back");
constexpr int kItems = 4;      // items that the load warp may be ahead
constexpr int kMostMixed = 8;  // tiles of an item in which rows see different keys: at most 6
constexpr int kSharedBytes = 3 * 1024;
// A row's reference is such that its largest weight is 2^kHeadroom when it moves, and moves when one exceeds 2^kSlack.  A
// call has less than 2^18 keys (check_args), so a row's weights add up to 1/2 at most and no finite V overflows the sums that
// are divided by them in the end.  What that costs lies at the other end: weights below 2^-126, 2^-99 of the largest, are zero.
constexpr float kHeadroom = -27.f, kSlack = -19.f;
static_assert((INT32_MAX / 8192) >> 18 == 0, "weights of 2^18 keys at most");

// Codes of the status word (waits that ran out).
enum : uint32_t { kTimeoutSoftmax = 61, kTimeoutLoad = 62, kTimeoutMma = 63, kTimeoutHelper = 64 };

struct Call {
    void *out;
    int64_t out_ld;
    const int32_t *offsets;  // or null: one sequence
    uint32_t *status;        // device status word, or null
    int32_t n_seqs, total, window;
    int32_t kv_heads, group, tokens;  // tokens of a row tile: kTile / group
    int32_t causal, out_bf16;
    float factor;            // |scale| in powers of two, above zero: a masked score of -infinity stays one
    uint32_t flip;           // sign bit of a negative scale
};

template <int D>
struct Cfg {
    static constexpr int kOperand = kTile * D * 2;  // a row tile of Q, a tile of K or V
    static constexpr int kKs = D == 128 ? 2 : 4, kVs = D == 128 ? 3 : 4;
    static constexpr int kKAt = 2 * kOperand, kVAt = kKAt + kKs * kOperand, kBarAt = kVAt + kVs * kOperand;
    static constexpr int kSmem = kBarAt + kSharedBytes;
    // Columns of tensor memory: scores from 0, and behind them the weights, where they fit (else over the scores), and the sums.
    static constexpr bool kApart = 2 * (kTile + kTile / 2 + D) <= 512;
    static constexpr int kWeightCols = kApart ? 2 * kTile : 0, kWeightStep = kApart ? kTile / 2 : kTile;
    static constexpr int kOutCols = kApart ? 3 * kTile : 2 * kTile;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Two row tiles of a sequence, for one KV head.
struct Item {
    int32_t begin, len;  // of the sequence: first row, tokens (0: no more items)
    int32_t token0, head;
    int32_t lo, hi;      // keys that any row sees
    int32_t all_lo, all_hi;  // keys that every row sees
    int32_t first[2], end[2];  // key tiles that a row tile uses: [first, end), none if it has no tokens

    NVFP4_DEVINL int tiles() const { return (hi - lo + kTile - 1) >> kTileShift; }
    NVFP4_DEVINL bool uses(int t, int tile) const { return tile >= first[t] && tile < end[t]; }
    NVFP4_DEVINL bool mixed(int tile) const
    {
        const int key0 = lo + tile * kTile;
        return key0 < all_lo || key0 + kTile > all_hi;
    }
};

struct Shared {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], v_ready[4];
    uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2][2], sums_ready[2], o_full[2], o_free[2], s_free[2], pv_done[2], drain;
    uint64_t item_full[kItems], item_empty[kItems], scanned[kItems];
    Item item[kItems];
    uint32_t bad[kItems];                         // whether the item has bad keys
    uint32_t bad_keys[kItems][kMostMixed][4];     // bit by key, of the item's mixed tiles in order
    float sum[2][kTile];  // of the weights, by row
    uint32_t tmem;
};
static_assert(sizeof(Shared) <= kSharedBytes, "barriers");

// tc::mbar_wait with the loop out of line: the roles share one instruction cache of some 32 KB.
NVFP4_DEVINL bool wait(uint64_t *bar, uint32_t parity) { return tc::mbar_wait_a(tc::smem_addr(bar), parity); }

// Keys [lo, hi) of a sequence that its token sees.
NVFP4_DEVINL void key_range(const Call &c, int len, int token, int *lo, int *hi)
{
    *lo = c.window > 0 ? max(0, token + 1 - c.window) : 0;
    *hi = c.causal ? token + 1 : len;
}

// ---------------------------------------------------------------------------
// Load warp
// ---------------------------------------------------------------------------

// Items of a call in order: 32 sequences after the other (each chunk of them is looked at once, however many there are),
// and among those the heaviest first: by place in the sequence (a sequence's last ones first), then by sequence, then by
// head; without a causal mask, where all items of a sequence cost the same, by sequence, the longest first.
struct Cursor {
    int level, chunk;  // place, and 32 sequences of which lane i holds the i-th
    int begin, len, places;  // the lane's: places of two row tiles
    uint32_t with;     // lanes whose sequence has the level's place
    uint32_t pos;      // number of the first item of the level (a call has less than 2^31)
    uint32_t rank;     // by sequence: places and lane of the one at hand
    int reached;       // end of the sequences so far
    bool descended;    // whether an offset did

    __device__ __noinline__ void load(const Call &c, int lane)
    {
        const int b = chunk + lane;
        int end = c.total;
        begin = b < c.n_seqs ? 0 : c.total;
        bool ok = true;
        if (c.offsets && b < c.n_seqs) {
            begin = c.offsets[b];
            end = c.offsets[b + 1];
            ok = begin >= 0 && end >= begin && end <= c.total;
        }
        // where offsets descend, later sequences may lie on earlier ones: the rows belong to the first
        descended |= __any_sync(0xFFFFFFFFu, !ok);
        if (__builtin_expect(descended, 0)) {
#pragma unroll 1
            for (int i = 0; i < 32; ++i) {
                ok = ok && (lane != i || begin >= reached);
                reached = max(reached, __shfl_sync(0xFFFFFFFFu, ok ? end : 0, i));
            }
        } else {
            reached = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)end);
        }
        if (!ok && blockIdx.x == 0)
            kv::report_index(c.status, kStatusPromptOffsets);
        len = ok ? end - begin : 0;
        places = (int)((uint32_t)(len + 2 * c.tokens - 1) / (2u * c.tokens));
    }
    // To the chunk's first item.
    NVFP4_DEVINL void open(const Call &c, int lane)
    {
        load(c, lane);
        level = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)places) - 1;
        with = __ballot_sync(0xFFFFFFFFu, places > level);
        rank = 0xFFFFFFFFu;
        next_rank(lane);
    }
    NVFP4_DEVINL void start()
    {
        chunk = -32;
        pos = rank = 0;
        reached = 0;
        descended = false;
        level = -1;
    }
    // The next sequence by length.
    NVFP4_DEVINL void next_rank(int lane)
    {
        const uint32_t mine = (uint32_t)places << 5 | (31 - lane);
        rank = __reduce_max_sync(0xFFFFFFFFu, places > 0 && mine < rank ? mine : 0u);
    }
    // Item number `want` (not before the last one asked for); false if there are not as many.
    NVFP4_DEVINL bool find(const Call &c, int lane, uint32_t want, Item *it)
    {
        uint32_t k;
        int src, place;
#pragma unroll 1
        for (;;) {
            if (c.causal ? level < 0 : rank == 0) {
                if (chunk + 32 >= c.n_seqs)
                    return false;
                chunk += 32;
                open(c, lane);
                continue;
            }
            const uint32_t count = (c.causal ? __popc(with) : rank >> 5) * c.kv_heads;
            if (want < pos + count)
                break;
            if (c.causal) {
                // on by as many levels as have the same sequences, or to the one that has the item
                const int last = (int)__reduce_max_sync(0xFFFFFFFFu, places > level ? 0u : (unsigned)places);
                const uint32_t skip = min((uint32_t)(level - last + 1), (want - pos) / count);
                pos += skip * count;
                level -= (int)skip;
                with = __ballot_sync(0xFFFFFFFFu, places > level);
            } else {
                pos += count;
                next_rank(lane);
            }
        }
        k = want - pos;
        if (c.causal) {
            const uint32_t which = k / (uint32_t)c.kv_heads;
            k -= which * c.kv_heads;
            // the lane that has `which` others before it
            const uint32_t before = with & ((1u << lane) - 1);
            src = __ffs(__ballot_sync(0xFFFFFFFFu, (with >> lane & 1) && __popc(before) == (int)which)) - 1;
            place = level;
        } else {
            src = 31 - (int)(rank & 31);
            place = (int)(k / (uint32_t)c.kv_heads);
            k -= place * c.kv_heads;
        }
        it->begin = __shfl_sync(0xFFFFFFFFu, begin, src);
        it->len = __shfl_sync(0xFFFFFFFFu, len, src);
        it->token0 = place * 2 * c.tokens;
        it->head = (int)k;
        const int last = min(it->token0 + 2 * c.tokens, it->len) - 1;
        key_range(c, it->len, it->token0, &it->lo, &it->all_hi);
        key_range(c, it->len, last, &it->all_lo, &it->hi);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int token0 = it->token0 + t * c.tokens;
            int lo, hi, unused;
            key_range(c, it->len, token0, &lo, &unused);
            key_range(c, it->len, min(token0 + c.tokens, it->len) - 1, &unused, &hi);
            it->first[t] = (lo - it->lo) >> kTileShift;
            it->end[t] = token0 < it->len ? (hi - it->lo + kTile - 1) >> kTileShift : 0;
        }
        return true;
    }
};

NVFP4_DEVINL void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

template <int D>
NVFP4_DEVINL bool load_role(const Call &c, const CUtensorMap *q_map, const CUtensorMap *k_map, const CUtensorMap *v_map,
                            Shared *sh, uint32_t smem, int lane)
{
    using C = Cfg<D>;
    Cursor cur;
    cur.start();
    uint32_t loaded = 0, q_items = 0, q_items_1 = 0;  // tiles of K (and V), and queries of row tile 0 and 1
    const uint32_t ctas = gridDim.x;
    bool ok = true;
    // one operand: waits for its place (round: how often that was used), and copies it in blocks of 64 elements
    const auto load = [&](const CUtensorMap *map, uint64_t *full, uint64_t *empty, uint32_t round, uint32_t at, uint32_t bytes,
                          int head, int row) {
        ok = ok && (round == 0 || wait(empty, (round - 1) & 1));
        if (!ok)
            return;
        tc::mbar_arrive_expect_tx(full, bytes);
#pragma unroll 1
        for (int b = 0; b < D; b += 64)
            tma_load_3d(at + b * (kTile * 2), map, tc::smem_addr(full), b, head, row);
    };
    for (uint32_t n = 0;; ++n) {
        Item it;
        const bool any = cur.find(c, lane, n * ctas + (n & 1 ? ctas - 1 - blockIdx.x : blockIdx.x), &it);
        const uint32_t slot = n % kItems;
        if (lane == 0) {
            ok = n < kItems || wait(&sh->item_empty[slot], (n / kItems - 1) & 1);
            if (!any)
                it.len = 0;
            sh->item[slot] = it;
            sh->bad[slot] = 0;
            tc::mbar_arrive(&sh->item_full[slot]);
            const int tiles = any ? it.tiles() : 0;
#pragma unroll 1
            for (int tile = 0; tile < tiles && ok; ++tile, ++loaded) {
                const int row = it.begin + it.lo + tile * kTile;
                const uint32_t k = loaded % C::kKs, v = loaded % C::kVs;
                load(k_map, &sh->k_full[k], &sh->k_empty[k], loaded / C::kKs, smem + C::kKAt + k * C::kOperand, C::kOperand, it.head, row);
                // the first keys do not wait until the queries before are done with
#pragma unroll 1
                for (int t = 0; tile == 0 && t < 2 && it.token0 + t * c.tokens < it.len; ++t) {
                    load(q_map, &sh->q_full[t], &sh->q_empty[t], t ? q_items_1 : q_items, smem + t * C::kOperand,
                         c.group * c.tokens * D * 2, it.head * c.group, it.begin + it.token0 + t * c.tokens);
                    q_items += 1 - t;
                    q_items_1 += t;
                }
                load(v_map, &sh->v_full[v], &sh->v_empty[v], loaded / C::kVs, smem + C::kVAt + v * C::kOperand, C::kOperand, it.head, row);
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!any || !ok)
            break;
    }
    // Nothing is in flight when the warp leaves: without a timeout the other warps have waited for every load; with one,
    // the waits for the last loads run out or not, but no load is younger than they are.
    if (lane == 0 && !ok) {
#pragma unroll 1
        for (uint32_t i = loaded > C::kKs ? loaded - C::kKs : 0; i < loaded; ++i)
            wait(&sh->k_full[i % C::kKs], (i / C::kKs) & 1);
#pragma unroll 1
        for (uint32_t i = loaded > C::kVs ? loaded - C::kVs : 0; i < loaded; ++i)
            wait(&sh->v_full[i % C::kVs], (i / C::kVs) & 1);
    }
    return ok;
}

// ---------------------------------------------------------------------------
// MMA warp
// ---------------------------------------------------------------------------

// Operand descriptors (swizzled rows of 128 bytes, in groups of 8) by their low word: start address / 16 and leading offset,
// which is that between 64-element column blocks where the rows are the reduction.
NVFP4_DEVINL uint32_t row_desc(uint32_t addr) { return (addr & 0x3FFFFu) >> 4 | 1u << 16; }
NVFP4_DEVINL uint32_t column_desc(uint32_t addr) { return (addr & 0x3FFFFu) >> 4 | (uint32_t)(kTile * 128 >> 4) << 16; }
NVFP4_DEVINL uint64_t desc(uint32_t low)
{
    constexpr uint32_t high = 1024 >> 4 | 1u << 14 | 2u << 29;
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "n"(high));
    return d;
}

// One thread issues every product, in the order
//     S0(0) S1(0)  then for each key tile i:  PV0(i) S0(i+1) PV1(i) S1(i+1),
// so that one row tile's products run while the other is in its softmax.  Products of one thread run in the order of
// issue, which lets S(i+1) overwrite the scores that PV(i) reads as weights.  (A thread for each row tile: both came
// to wait for their softmax at the same time, 1.98 ms where this took 1.81; the two taking turns 1.87 where it took
// 1.70; a thread for the scores and one for the outputs 2.03.)
template <int D>
NVFP4_DEVINL bool mma_role(const Call &c, Shared *sh, uint32_t smem, uint32_t tmem)
{
    using C = Cfg<D>;
    constexpr uint32_t score_idesc = tc::idesc_f16kind(kTile, kTile, 1);
    constexpr uint32_t out_idesc = tc::idesc_f16kind(kTile, D, 1) | 1u << 16;  // B transposed
    uint32_t ks = 0, vs = 0, items[2] = {0, 0}, mine[2] = {0, 0};  // tiles of K and V so far, the row tiles' items and products P V
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kItems;
        if (!(ok = wait(&sh->item_full[slot], (n / kItems) & 1)))
            break;
        const Item it = sh->item[slot];
        tc::mbar_arrive(&sh->item_empty[slot]);
        if (it.len == 0)
            break;
        const int tiles = it.tiles();
        // (one place in the code for the first scores and the others)
#pragma unroll 1
        for (int i = -1; i < tiles && ok; ++i) {
            const uint32_t v_slot = vs % C::kVs, v_phase = (vs / C::kVs) & 1;
            const uint32_t v = column_desc(smem + C::kVAt + v_slot * C::kOperand);
            const bool more = i + 1 < tiles;
            if (i >= 0) {
                ++vs;
                ok = wait(&sh->v_full[v_slot], v_phase) && wait(&sh->v_ready[v_slot], v_phase);
            }
            if (more)
                ok = ok && wait(&sh->k_full[ks % C::kKs], (ks / C::kKs) & 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (i >= 0 && it.uses(t, i)) {
                    // the item before has been read out
                    if (i == it.first[t] && items[t] > 1)
                        ok = ok && wait(&sh->o_free[t], items[t] & 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && wait(&sh->p_ready[t][h], mine[t] & 1);
                        if (!ok)
                            break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int j = 0; j < kTile / 32; ++j)
                            tc::mma_f16_ts(tmem + C::kOutCols + t * D, tmem + t * kTile + h * (kTile / 4) + 8 * j,
                                           desc(v + ((h * (kTile / 32) + j) * 2048 >> 4)), out_idesc,
                                           i > it.first[t] || h > 0 || j > 0);
                    }
                    if (!ok)
                        break;
                    ++mine[t];
                    if (i + 1 == it.end[t])
                        tc::mma_commit(&sh->o_full[t]);
                }
                if (t == 1 && i >= 0)
                    tc::mma_commit(&sh->v_empty[v_slot]);
                if (more && it.uses(t, i + 1)) {
                    if (i + 1 == it.first[t])
                        ok = ok && wait(&sh->q_full[t], items[t]++ & 1);
                    if (!ok)
                        break;
                    const uint32_t k = row_desc(smem + C::kKAt + (ks % C::kKs) * C::kOperand), q = row_desc(smem + t * C::kOperand);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        const uint32_t at = ((d / 4) * (kTile * 128) + (d % 4) * 32) >> 4;
                        tc::mma_bf16_ss(tmem + t * kTile, desc(q + at), desc(k + at), score_idesc, d > 0);
                    }
                    tc::mma_commit(&sh->s_full[t]);
                    if (i + 2 == it.end[t])
                        tc::mma_commit(&sh->q_empty[t]);
                }
            }
            if (more)
                tc::mma_commit(&sh->k_empty[ks++ % C::kKs]);
        }
    }
    // nothing of this thread's is in flight when it leaves
    tc::mma_commit(&sh->drain);
    return wait(&sh->drain, 0) && ok;
}

// The same where the weights have columns of their own (heads of 64): a row tile's next scores are made as soon as its
// softmax has read the last ones, in the order
//     S0(s+1) PV1(s-1) S1(s+1) PV0(s)
// of key tiles s, on through all items.  The scores are not waited for at once, so that one commit tells of them and of the
// other row tile's sums: two stops a step instead of four.  5 images of 577 to 2305 tokens 65 -> 62 us (with four stops 64), a
// window of 1024 57.6 -> 57.2.
template <int D>
NVFP4_DEVINL bool mma_apart_role(const Call &c, Shared *sh, uint32_t smem, uint32_t tmem)
{
    using C = Cfg<D>;
    constexpr uint32_t score_idesc = tc::idesc_f16kind(kTile, kTile, 1);
    constexpr uint32_t out_idesc = tc::idesc_f16kind(kTile, D, 1) | 1u << 16;  // B transposed
    // of a step, for row tile t: bit 3 t that it uses the keys, 3 t + 1 that they are its first, 3 t + 2 its last
    uint32_t flags[3] = {0, 0, 0};  // of the steps before the last one, of the last one, and of the next one
    uint32_t items[2] = {0, 0}, scored[2] = {0, 0}, summed[2] = {0, 0}, outs[2] = {0, 0};  // of the row tiles, so far
    bool ok = true;
    const auto scores = [&](int t, uint32_t step, uint32_t f) {
        f >>= 3 * t;
        if (!(f & 1))
            return;
        ok = ok && (scored[t] == 0 || wait(&sh->s_free[t], (scored[t] - 1) & 1));
        ++scored[t];
        if (f & 2)
            ok = ok && wait(&sh->q_full[t], items[t]++ & 1);
        if (!ok)
            return;
        tc::fence_after_sync();
        const uint32_t k = row_desc(smem + C::kKAt + (step % C::kKs) * C::kOperand), q = row_desc(smem + t * C::kOperand);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            const uint32_t at = ((d / 4) * (kTile * 128) + (d % 4) * 32) >> 4;
            tc::mma_bf16_ss(tmem + t * kTile, desc(q + at), desc(k + at), score_idesc, d > 0);
        }
    };
    const auto sums = [&](int t, uint32_t step, uint32_t f) {
        f >>= 3 * t;
        if (!(f & 1))
            return;
        const uint32_t v_slot = step % C::kVs, v_phase = (step / C::kVs) & 1;
        const uint32_t v = column_desc(smem + C::kVAt + v_slot * C::kOperand);
        ok = ok && wait(&sh->v_full[v_slot], v_phase) && wait(&sh->v_ready[v_slot], v_phase);
        // the item before has been read out
        if (f & 2 && outs[t]++ > 0)
            ok = ok && wait(&sh->o_free[t], outs[t] & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ok = ok && wait(&sh->p_ready[t][h], summed[t] & 1);
            if (!ok)
                return;
            tc::fence_after_sync();
#pragma unroll
            for (int j = 0; j < kTile / 32; ++j)
                tc::mma_f16_ts(tmem + C::kOutCols + t * D, tmem + C::kWeightCols + t * C::kWeightStep + h * (kTile / 4) + 8 * j,
                               desc(v + ((h * (kTile / 32) + j) * 2048 >> 4)), out_idesc, !(f & 2) || h > 0 || j > 0);
        }
        ++summed[t];
    };
    const auto commit = [&](int t, uint32_t fs, uint32_t fp) {  // scores of t, and sums of the other
        fs >>= 3 * t;
        fp >>= 3 * (1 - t);
        if (!ok)
            return;
        if (fs & 1)
            tc::mma_commit(&sh->s_full[t]);
        if (fp & 1)
            tc::mma_commit(&sh->pv_done[1 - t]);
        if ((fs & 5) == 5)
            tc::mma_commit(&sh->q_empty[t]);
        if ((fp & 5) == 5)
            tc::mma_commit(&sh->o_full[1 - t]);
    };
    Item it;
    int tile = 0, tiles = 0, drain = 0;
    uint32_t n = 0;
#pragma unroll 1
    for (uint32_t step = 0; ok && drain < 2; ++step) {  // the next one
        if (drain == 0 && tile == tiles) {
            const uint32_t slot = n % kItems;
            if (!(ok = wait(&sh->item_full[slot], (n / kItems) & 1)))
                break;
            it = sh->item[slot];
            tc::mbar_arrive(&sh->item_empty[slot]);
            ++n;
            tile = 0;
            tiles = it.len ? it.tiles() : 0;
        }
        flags[2] = 0;
        const bool more = drain == 0 && tiles > 0;
        if (more) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (it.uses(t, tile))
                    flags[2] |= (1u | (tile == it.first[t] ? 2u : 0u) | (tile + 1 == it.end[t] ? 4u : 0u)) << 3 * t;
            ++tile;
            ok = wait(&sh->k_full[step % C::kKs], (step / C::kKs) & 1);
        } else {
            ++drain;
        }
        scores(0, step, flags[2]);
        sums(1, step - 2, flags[0]);
        commit(0, flags[2], flags[0]);
        if (step >= 2 && ok)
            tc::mma_commit(&sh->v_empty[(step - 2) % C::kVs]);
        scores(1, step, flags[2]);
        sums(0, step - 1, flags[1]);
        commit(1, flags[2], flags[1]);
        if (more && ok)
            tc::mma_commit(&sh->k_empty[step % C::kKs]);
        flags[0] = flags[1];
        flags[1] = flags[2];
    }
    // nothing of this thread's is in flight when it leaves
    tc::mma_commit(&sh->drain);
    return wait(&sh->drain, 0) && ok;
}

// ---------------------------------------------------------------------------
// Helper warps
// ---------------------------------------------------------------------------

// All ones in the halves of a word of two bf16 that are infinities or NaN.
NVFP4_DEVINL uint32_t not_finite(uint32_t w)
{
    const uint32_t m = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    return (m >> 15) * 0xFFFFu;
}

// Writes zeros in place of what is not finite, and returns in which of four rows there was any (8 lanes to a row).
__device__ __noinline__ uint32_t take_out(uint32_t at, uint4 w, uint4 m, bool any, uint32_t lanes)
{
    if (any)
        tc::sts128(at, make_uint4(w.x & ~m.x, w.y & ~m.y, w.z & ~m.z, w.w & ~m.w));
    uint32_t rows = 0;
    for (int k = 0; k < 4; ++k)
        rows |= (lanes >> 8 * k & 0xFFu ? 1u : 0u) << k;
    return rows;
}

// Bits j of a word for keys first + j that lie in [lo, hi).
NVFP4_DEVINL uint32_t range_bits(int first, int lo, int hi)
{
    const int a = max(lo - first, 0), b = min(hi - first, 32);
    return a >= b ? 0u : (0xFFFFFFFFu << a) & (0xFFFFFFFFu >> (32 - b));
}

// Adds the infinities and NaN of V that a row sees (keys [lo, hi)) in the tiles from which they were taken out to its
// output, which the thread has stored.  v: of the sequence's first token.
template <int D>
__device__ __noinline__ void add_not_finite(const Item *it, const uint32_t (*bad_keys)[4], const uint16_t *v, int64_t v_ld, int lo,
                                            int hi, void *out, int out_bf16)
{
    int mixed = 0;
#pragma unroll 1
    for (int i = 0; i < it->tiles(); ++i) {
        if (!it->mixed(i))
            continue;
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
            const int key0 = it->lo + i * kTile + 32 * w;
#pragma unroll 1
            for (uint32_t keys = bad_keys[mixed][w] & range_bits(key0, lo, hi); keys; keys &= keys - 1) {
                const uint16_t *src = v + (int64_t)(key0 + __ffs(keys) - 1) * v_ld;
#pragma unroll 1
                for (int d = 0; d < D; ++d) {
                    const float e = __uint_as_float((uint32_t)src[d] << 16);
                    if (isfinite(e))
                        continue;
                    if (out_bf16) {
                        uint16_t *o = static_cast<uint16_t *>(out) + d;
                        *o = f32_to_bf16(__uint_as_float((uint32_t)*o << 16) + e);
                    } else {
                        static_cast<float *>(out)[d] += e;
                    }
                }
            }
        }
        ++mixed;
    }
}

NVFP4_DEVINL void store_32_bytes(void *p, const uint32_t (&w)[8], bool aligned_32)
{
    if (aligned_32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// The output rows of a row tile of an item, 32 of them (`warp`, a row to a lane): sums / (sum of the weights).
template <int D>
NVFP4_DEVINL void store_rows(const Call &c, const Item *it, const uint32_t (*bad_keys)[4], bool bad, const uint16_t *v, int64_t v_ld,
                             int t, int r, int my_token, int my_head, float sum, uint32_t out)
{
    const int token = it->token0 + t * c.tokens + my_token;
    const bool live = my_token < c.tokens && token < it->len;
    const float inv = 1.f / sum;
    const int width = c.out_bf16 ? 2 : 4;
    uint8_t *const dst = static_cast<uint8_t *>(c.out) +
                         ((int64_t)(it->begin + token) * c.out_ld + (int64_t)(it->head * c.group + my_head) * D) * width;
    const bool aligned_32 = (reinterpret_cast<uintptr_t>(c.out) | (uintptr_t)c.out_ld * width) % 32 == 0;
#pragma unroll 1
    for (int q = 0; q < D; q += 16) {
        uint32_t x[16];
        tc::tmem_ld_32x32b_x16(out + q, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            asm volatile("" : "+r"(x[j]));
            x[j] = __float_as_uint(__uint_as_float(x[j]) * inv);
        }
        // 32 bytes a store: a row's neighbours in the warp lie in other lines, and each line costs the store a clock
        if (live && c.out_bf16) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = f32x2_to_bf16x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
            store_32_bytes(dst + q * 2, w, aligned_32);
        } else if (live) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = x[8 * k + j];
                store_32_bytes(dst + (q + 8 * k) * 4, w, aligned_32);
            }
        }
        __syncwarp();
    }
    if (__builtin_expect(bad && live, 0)) {
        int lo, hi;
        key_range(c, it->len, token, &lo, &hi);
        add_not_finite<D>(it, bad_keys, v + (int64_t)it->begin * v_ld + (int64_t)it->head * D, v_ld, lo, hi, dst, c.out_bf16);
    }
    __syncwarp();
}

// Whether a phase is complete, without waiting.
NVFP4_DEVINL bool complete(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(tc::smem_addr(bar)), "r"(parity)
                 : "memory");
    return __all_sync(0xFFFFFFFFu, ok != 0);
}

// Looks through the items' tiles of V, and writes the output rows of the items that are done, whichever comes first: neither
// may wait for the other (the tiles of the next items come before the last products of this one).
template <int D>
NVFP4_DEVINL bool helper_role(const Call &c, const uint16_t *v, int64_t v_ld, Shared *sh, uint32_t smem, uint32_t tmem, int warp, int lane)
{
    using C = Cfg<D>;
    const int r = 32 * warp + lane, my_token = r / c.group, my_head = r - my_token * c.group;
    uint32_t n = 0, vs = 0;               // the item whose tiles are looked through, and tiles so far
    int tile = 0, mixed = 0;
    bool more = true;
    uint32_t rows[2] = {0, 0}, done[2] = {0, 0}, freed = 0;  // the items whose rows are written next, those written of each row tile
    uint32_t last = 0xFFFFFFFFu;          // the item that marks the end
    uint64_t idle = 0;
    while (freed < last) {
        bool progress = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t slot = rows[t] % kItems;
            if (rows[t] >= last || !complete(&sh->item_full[slot], (rows[t] / kItems) & 1))
                continue;
            const Item *const it = &sh->item[slot];
            if (it->len == 0) {
                last = rows[t];
                continue;
            }
            if (it->end[t] > 0) {
                if (!complete(&sh->o_full[t], done[t] & 1) || !complete(&sh->sums_ready[t], done[t] & 1) ||
                    !complete(&sh->scanned[slot], (rows[t] / kItems) & 1))
                    continue;
                tc::fence_after_sync();
                store_rows<D>(c, it, sh->bad_keys[slot], sh->bad[slot] != 0, v, v_ld, t, r, my_token, my_head, sh->sum[t][r],
                              tmem + C::kOutCols + t * D + ((uint32_t)(32 * warp) << 16));
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&sh->o_free[t]);
                ++done[t];
            }
            ++rows[t];
            progress = true;
        }
        for (; freed < min(rows[0], rows[1]); ++freed) {
            if (lane == 0)
                tc::mbar_arrive(&sh->item_empty[freed % kItems]);
        }
        const uint32_t slot = n % kItems, v_slot = vs % C::kVs;
        if (more && complete(&sh->item_full[slot], (n / kItems) & 1)) {
            const Item *const it = &sh->item[slot];
            if (it->len == 0) {
                more = false;
            } else if (tile == it->tiles()) {
                if (lane == 0)
                    tc::mbar_arrive(&sh->scanned[slot]);
                ++n;
                tile = mixed = 0;
                progress = true;
            } else if (complete(&sh->v_full[v_slot], (vs / C::kVs) & 1)) {
                if (it->mixed(tile)) {
                    // 32 rows of the tile, four at a time; 8 lanes to 128 bytes of a row
                    const uint32_t at = smem + C::kVAt + v_slot * C::kOperand + warp * 32 * 128 + lane * 16;
                    uint32_t bad = 0;
#pragma unroll 1
                    for (int b = 0; b < D / 64; ++b) {
#pragma unroll 4
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t a = at + b * kTile * 128 + k * 512;
                            const uint4 w = tc::lds128(a);
                            const uint4 m = make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w));
                            const bool any = (m.x | m.y | m.z | m.w) != 0;
                            const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, any);
                            if (lanes)
                                bad |= take_out(a, w, m, any, lanes) << 4 * k;
                        }
                    }
                    // keys that some row sees
                    const int key0 = it->lo + tile * kTile + warp * 32, some = it->hi - key0;
                    bad &= some <= 0 ? 0u : some >= 32 ? 0xFFFFFFFFu : (1u << some) - 1;
                    if (lane == 0) {
                        sh->bad_keys[slot][mixed][warp] = bad;
                        if (bad)
                            sh->bad[slot] = 1;
                    }
                    ++mixed;
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0)
                    tc::mbar_arrive(&sh->v_ready[v_slot]);
                ++tile;
                ++vs;
                progress = true;
            }
        }
        if (progress) {
            idle = 0;
        } else {
            const uint64_t now = tc::globaltimer();
            if (idle == 0)
                idle = now;
            if (__any_sync(0xFFFFFFFFu, now - idle > tc::kWaitLimitNs))
                return false;
            __nanosleep(20);
        }
    }
    return true;
}

// ---------------------------------------------------------------------------
// Softmax warps
// ---------------------------------------------------------------------------

// Scores of a tile some of whose keys some row does not see (the row sees [lo, hi) of it), or which a negative factor
// turns round: rewritten in tensor memory, 32 keys at a time and only where there is something to do.
__device__ __noinline__ void mask_scores(uint32_t scores, int lo, int hi, uint32_t flip)
{
#pragma unroll 1
    for (int q = 0; q < kTile; q += 32, lo -= 32, hi -= 32) {
        if (__all_sync(0xFFFFFFFFu, lo <= 0 && hi >= 32 && flip == 0))
            continue;
        uint32_t x[32];
        const uint32_t n = max(hi - lo, 0);
        if (__any_sync(0xFFFFFFFFu, hi > 0 && lo < 32)) {
            tc::tmem_ld_32x32b_x32(scores + q, x);
            tc::tmem_ld_wait();
            settle(x);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = (uint32_t)(j - lo) < n ? x[j] ^ flip : 0xFF800000u;  // -infinity
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = 0xFF800000u;
        }
        tc::tmem_st_32x32b_x32(scores + q, x);
    }
    tc::tmem_st_wait();
}

// Multiplies the row's sums so far.
template <int D>
NVFP4_DEVINL void rescale(uint32_t out, float shrink)
{
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
    tc::tmem_st_wait();
}

// A row's reference (what is taken from its scores), and the sum of its weights.
struct RowState {
    float top, sum;
};

// Weights of a tile's keys.  signals: of one lane of each warp.  begun: the row has sums already.  mine: the row tile's key
// tiles before.  False if a wait ran out.
template <int D>
NVFP4_DEVINL bool tile_weights(Shared *sh, int t, uint32_t scores, uint32_t weights, uint32_t out, bool signals, bool begun,
                               uint32_t mine, float f, RowState &row)
{
    bool ok = true;
    uint32_t s[4][32];  // first the largest
#pragma unroll
    for (int q = 0; q < 4; ++q)
        tc::tmem_ld_32x32b_x32(scores + 32 * q, s[q]);
    tc::tmem_ld_wait();
#pragma unroll
    for (int q = 0; q < 4; ++q)
        settle(s[q]);
    if (Cfg<D>::kApart) {
        tc::fence_before_sync();
        __syncwarp();
        if (signals)
            tc::mbar_arrive(&sh->s_free[t]);
    }
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            m[q] = max3(m[q], __uint_as_float(s[q][j]), __uint_as_float(s[q][j + 1]));
    }
    const float largest = max3(fmaxf(m[0], m[1]), m[2], m[3]) * f;
    if (Cfg<D>::kApart && mine > 0) {
        ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&sh->pv_done[t], (mine - 1) & 1));
        tc::fence_after_sync();
    }
    const bool over = largest - row.top > kSlack;  // (true for the first reference, false for a NaN)
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, over), 0)) {
        // move the row's reference, and with it what was summed up (the tile before's products are done: these
        // scores came after them)
        const float next = over ? largest - kHeadroom : row.top;
        const float shrink = over && row.top != -INFINITY ? ex2(row.top - next) : 1.f;
        row.top = next;
        row.sum *= shrink;
        if (begun && __any_sync(0xFFFFFFFFu, shrink != 1.f))
            rescale<D>(out, shrink);
    }
    const float add = row.top == -INFINITY ? 0.f : -row.top;
    const uint64_t f2 = pack2(f, f), add_2 = pack2(add, add);
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // halves of the keys: the product of the first begins meanwhile
        uint64_t l2[2] = {0, 0};
#pragma unroll
        for (int q = 2 * h; q < 2 * h + 2; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 e = unpack2(fma2(
                    pack2(__uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1])), f2, add_2));
                const float a = ex2(e.x), b = ex2(e.y);
                l2[j & 1] = add2(l2[j & 1], pack2(a, b));
                p[j] = f32x2_to_bf16x2(a, b);
            }
            tc::tmem_st_32x32b_x16(weights + 16 * q, p);
        }
        const float2 l = unpack2(add2(l2[0], l2[1]));
        row.sum += l.x + l.y;
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (signals)
            tc::mbar_arrive(&sh->p_ready[t][h]);
    }
    return ok;
}

template <int D>
NVFP4_DEVINL bool softmax_role(const Call &c, Shared *sh, uint32_t tmem, int tid)
{
    using C = Cfg<D>;
    const int t = tid / 128, r = tid % 128;  // row tile, and row of it: its lane of tensor memory
    const uint32_t lanes = (uint32_t)(r & ~31) << 16;
    const uint32_t scores = tmem + t * kTile + lanes, out = tmem + C::kOutCols + t * D + lanes;
    const int my_token = r / c.group + t * c.tokens;
    const bool has_token = r < c.tokens * c.group;
    bool ok = true;
    uint32_t mine = 0, items = 0;  // the row tile's key tiles and items so far
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kItems;
        ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&sh->item_full[slot], (n / kItems) & 1));
        if (!ok)
            break;
        const int len = sh->item[slot].len, first = sh->item[slot].first[t], end = sh->item[slot].end[t];
        const int token = sh->item[slot].token0 + my_token;
        int key0 = sh->item[slot].lo + first * kTile;
        if (len == 0)
            break;
        // rows beyond the last one: no key is masked, and none has any weight
        int lo = 0, hi = INT32_MAX;
        const bool live = has_token && token < len;
        if (live)
            key_range(c, len, token, &lo, &hi);
        RowState row{live ? -INFINITY : 1e30f, 0.f};
        for (int i = first; i < end; ++i, ++mine, key0 += kTile) {
            ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&sh->s_full[t], mine & 1));
            if (!ok)
                break;
            tc::fence_after_sync();
            if (__builtin_expect(!__all_sync(0xFFFFFFFFu, c.flip == 0 && key0 >= lo && key0 + kTile <= hi), 0))
                mask_scores(scores, lo - key0, hi - key0, c.flip);
            ok = tile_weights<D>(sh, t, scores, tmem + C::kWeightCols + t * C::kWeightStep + lanes, out, r % 32 == 0, i > first,
                                 mine, c.factor, row);
            if (!ok)
                break;
        }
        if (end > 0 && ok) {
            // (the helper warps have read the item before's sums)
            ok = __all_sync(0xFFFFFFFFu, items == 0 || tc::mbar_wait(&sh->o_free[t], (items - 1) & 1));
            sh->sum[t][r] = row.sum;
            ++items;
        }
        __syncwarp();
        if (r % 32 == 0) {
            if (end > 0)
                tc::mbar_arrive(&sh->sums_ready[t]);
            tc::mbar_arrive(&sh->item_empty[slot]);
        }
    }
    return ok;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, Call c, const uint16_t *v, int64_t v_ld)
{
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared *const sh = reinterpret_cast<Shared *>(smem_raw + C::kBarAt);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0), lane = tid % 32;

    tc::griddep_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&sh->k_full[i], 1);
            tc::mbar_init(&sh->v_full[i], 1);
            tc::mbar_init(&sh->k_empty[i], 1);
            tc::mbar_init(&sh->v_empty[i], 1);
            tc::mbar_init(&sh->v_ready[i], 4);
        }
        for (int t = 0; t < 2; ++t) {
            tc::mbar_init(&sh->q_full[t], 1);
            tc::mbar_init(&sh->q_empty[t], 1);
            tc::mbar_init(&sh->s_full[t], 1);
            tc::mbar_init(&sh->o_free[t], 4);
            tc::mbar_init(&sh->sums_ready[t], 4);
            tc::mbar_init(&sh->o_full[t], 1);
            tc::mbar_init(&sh->s_free[t], 4);
            tc::mbar_init(&sh->pv_done[t], 1);
            for (int h = 0; h < 2; ++h)
                tc::mbar_init(&sh->p_ready[t][h], 4);
        }
        tc::mbar_init(&sh->drain, 1);
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(&sh->item_full[i], 1);
            tc::mbar_init(&sh->item_empty[i], 1 + 8 + 4);  // MMA thread, softmax warps, helper warps
            tc::mbar_init(&sh->scanned[i], 4);
        }
        tc::fence_mbar_init();
    }
    if (warp == kAllocWarp)
        tc::tmem_alloc(&sh->tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t smem = tc::smem_addr(smem_raw), tmem = sh->tmem;
    tc::griddep_wait();  // from here on, what the kernel before wrote is read, and what it reads may be written

    bool ok = true;
    uint32_t code = 0;
    if (warp < kLoadWarp) {
        take_regs<kSoftmaxRegs>();
        ok = softmax_role<D>(c, sh, tmem, tid);
        code = kTimeoutSoftmax;
    } else {
        give_regs<kOtherRegs>();
        if (warp == kLoadWarp) {
            ok = load_role<D>(c, &q_map, &k_map, &v_map, sh, smem, lane);
            code = kTimeoutLoad;
        } else if (warp == kMmaWarp) {
            if (elect_one()) {
                ok = C::kApart ? mma_apart_role<D>(c, sh, smem, tmem) : mma_role<D>(c, sh, smem, tmem);
                code = kTimeoutMma;
            }
            __syncwarp();
        } else if (warp >= kHelperWarp) {
            ok = helper_role<D>(c, v, v_ld, sh, smem, tmem, warp - kHelperWarp, lane);
            code = kTimeoutHelper;
        }
    }
    if (!ok)
        kv::report_timeout(c.status, code);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kAllocWarp)
        tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_args(const nvfp4_prompt_attention_args *a)
{
    if (!a || a->n_seqs < 0 || a->total < 0 || a->window < 0)
        return NVFP4_ERR_INVALID_ARG;
    if ((a->out_dtype != NVFP4_OUT_F32 && a->out_dtype != NVFP4_OUT_BF16) || (a->causal != 0 && a->causal != 1) ||
        (a->window > 0 && !a->causal) || !std::isfinite(a->scale * 1.4426950408889634f) || (!a->offsets && a->n_seqs != 1))
        return NVFP4_ERR_INVALID_ARG;
    if (a->head_dim != 64 && a->head_dim != 128)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (a->n_kv_heads < 1 || a->n_q_heads < 1 || a->n_q_heads > 8192 || a->n_q_heads % a->n_kv_heads != 0 ||
        a->n_q_heads / a->n_kv_heads > kMaxGroup || a->n_seqs > 65535 || a->total > INT32_MAX / 8192)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (a->total == 0 || a->n_seqs == 0)
        return NVFP4_OK;
    const int64_t q_width = (int64_t)a->n_q_heads * a->head_dim, kv_width = (int64_t)a->n_kv_heads * a->head_dim;
    const auto stride_ok = [&](int64_t ld, int64_t width) {
        return ld >= width && ld % 8 == 0 && ld <= (INT64_C(1) << 38) / 8;  // (a tensor map's stride is below 2^40 bytes)
    };
    if (!stride_ok(a->q_ld, q_width) || !stride_ok(a->k_ld, kv_width) || !stride_ok(a->v_ld, kv_width) ||
        !stride_ok(a->out_ld, q_width))
        return NVFP4_ERR_INVALID_ARG;
    if (!a->q || !a->k || !a->v || !a->out || !aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) ||
        !aligned(a->out, 16) || !aligned(a->offsets, 4))
        return NVFP4_ERR_INVALID_ARG;
    return NVFP4_OK;
}

template <int D>
cudaError_t launch(const nvfp4_prompt_attention_args &a, const Call &c, int num_sms, cudaStream_t stream)
{
    using C = Cfg<D>;
    static std::once_flag once[kMaxDevices];
    static cudaError_t results[kMaxDevices];
    const auto kernel = prompt_kernel<D>;
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
    // [row][head][element], 64 elements (128 bytes, swizzled) of some heads and rows at a time
    CUtensorMap q, k, v;
    if (!sk::make_head_map(&q, a.q, D, a.n_q_heads, a.total, a.q_ld, c.group, c.tokens) ||
        !sk::make_head_map(&k, a.k, D, a.n_kv_heads, a.total, a.k_ld, 1, kTile) ||
        !sk::make_head_map(&v, a.v, D, a.n_kv_heads, a.total, a.v_ld, 1, kTile))
        return cudaErrorInvalidValue;
    // no more CTAs than items there can be
    const int64_t items = ((int64_t)c.total / (2 * c.tokens) + c.n_seqs) * c.kv_heads;
    return launch_dependent(kernel, dim3((unsigned)(items < num_sms ? items : num_sms)), kThreads, C::kSmem, stream, q, k, v, c,
                            a.v, a.v_ld);
}

}  // namespace prompt
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int nvfp4_prompt_attention(const nvfp4_prompt_attention_args *args, void *workspace, size_t workspace_bytes,
                                      nvfp4_stream_t stream)
{
    int rc = prompt::check_args(args);
    if (rc != NVFP4_OK)
        return rc;
    if (workspace && !prompt::aligned(workspace, 16))
        return NVFP4_ERR_INVALID_ARG;
    if (workspace && workspace_bytes < kKvWorkspaceBytes)
        return NVFP4_ERR_WORKSPACE;
    if (args->total == 0 || args->n_seqs == 0)
        return NVFP4_OK;
    if (args->out == args->q || args->out == args->k || args->out == args->v)  // other CTAs read them after rows are written
        return NVFP4_ERR_INVALID_ARG;
    prompt::Call c;
    c.out = args->out;
    c.out_ld = args->out_ld;
    c.offsets = args->offsets;
    c.status = workspace ? reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + kStatusWordOffset) : nullptr;
    c.n_seqs = (int32_t)args->n_seqs;
    c.total = (int32_t)args->total;
    c.window = args->window > INT32_MAX ? 0 : (int32_t)args->window;
    c.kv_heads = args->n_kv_heads;
    c.group = args->n_q_heads / args->n_kv_heads;
    c.tokens = prompt::kTile / c.group;
    c.causal = args->causal;
    c.out_bf16 = args->out_dtype == NVFP4_OUT_BF16;
    c.factor = std::fmax(std::fabs(args->scale * 1.4426950408889634f), 0x1p-126f);
    c.flip = args->scale < 0.f ? 0x80000000u : 0u;
    int sms = 0;
    rc = current_num_sms(&sms);
    if (rc != NVFP4_OK)
        return rc;
    const cudaError_t e = args->head_dim == 64 ? prompt::launch<64>(*args, c, sms, (cudaStream_t)stream)
                                               : prompt::launch<128>(*args, c, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
