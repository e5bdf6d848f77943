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
//                   memory, the weights P go back there in bf16 as the A operand of the second product,
//                   over the scores.  A row's reference (an upper estimate of its largest score) moves
//                   only when 64 weights sum to more than 2^15, so there is no pass for the maximum.
//   warp 8          finds the items and loads Q, K and V by TMA.
//   warp 9          MMA issue.
//   warps 12-15     look through V tiles in which rows see different keys: an infinity or a NaN
//                   there would reach every row through 0 * inf, so it is taken out of the tile, and
//                   added at the end to the rows that do see it.
//
// Items are taken heaviest first (the last tokens of the sequences, then those before them), CTA c of P taking
// the c-th of every P, in alternating directions: for one long causal prompt every CTA then has the same
// number of keys to within a tile.  The lengths are on the device, so each CTA finds its items itself.
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
constexpr int kTile = 128;      // keys of a tile, rows of a row tile
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kAllocWarp = 10, kScanWarp = 12;
// Registers of a thread by role: what the launch gives every thread, shared out anew.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 176, kOtherRegs = 80;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= kThreads * kLaunchRegs,
              "setmaxnreg would wait for registers that nobody gives back");
constexpr int kItems = 4;      // items that the load warp may be ahead
constexpr int kMostMixed = 8;  // tiles of an item in which rows see different keys: at most 6
constexpr int kSharedBytes = 2048;
constexpr float kHeadroom = 7.f;
constexpr float kMostWeight = 0x1p15f;  // of the weights of half a tile, in sum

// Codes of the status word (waits that ran out).
enum : uint32_t { kTimeoutSoftmax = 61, kTimeoutLoad = 62, kTimeoutMma = 63, kTimeoutScan = 64 };

struct Call {
    void *out;
    int64_t out_ld;
    const int32_t *offsets;  // or null: one sequence
    uint32_t *status;        // device status word, or null
    int32_t n_seqs, total, window;
    int32_t kv_heads, group, tokens;  // tokens of a row tile: kTile / group
    int32_t causal, out_bf16;
    float scale_log2;        // scores in powers of two
};

template <int D>
struct Cfg {
    static constexpr int kOperand = kTile * D * 2;  // a row tile of Q, a tile of K or V
    static constexpr int kKs = D == 128 ? 2 : 4, kVs = D == 128 ? 3 : 4;
    static constexpr int kKAt = 2 * kOperand, kVAt = kKAt + kKs * kOperand, kBarAt = kVAt + kVs * kOperand;
    static constexpr int kSmem = kBarAt + kSharedBytes;
    static constexpr int kOutCols = 2 * kTile;  // of tensor memory, behind the scores
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Two row tiles of a sequence, for one KV head.
struct Item {
    int32_t begin, len;  // of the sequence: first row, tokens (0: no more items)
    int32_t token0, head;
    int32_t lo, hi;      // keys that any row sees
    int32_t all_lo, all_hi;  // keys that every row sees

    NVFP4_DEVINL int tiles() const { return (hi - lo + kTile - 1) / kTile; }
    NVFP4_DEVINL bool mixed(int tile) const
    {
        const int key0 = lo + tile * kTile;
        return key0 < all_lo || key0 + kTile > all_hi;
    }
};

struct Shared {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], v_ready[4];
    uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2][2], half_done[2], o_full[2], o_free[2], drain;
    uint64_t item_full[kItems], item_empty[kItems], scanned[kItems];
    Item item[kItems];
    uint32_t bad[kItems];                         // whether the item has bad keys
    uint32_t bad_keys[kItems][kMostMixed][4];     // bit by key, of the item's mixed tiles in order
    uint32_t tmem;
};
static_assert(sizeof(Shared) <= kSharedBytes, "barriers");

// Keys [lo, hi) of a sequence that its token sees.
NVFP4_DEVINL void key_range(const Call &c, int len, int token, int *lo, int *hi)
{
    *lo = c.window > 0 ? max(0, token + 1 - c.window) : 0;
    *hi = c.causal ? token + 1 : len;
}

// A row tile's share of an item: its tokens, and the key tiles [first, end) that any of them sees.
struct Part {
    int token0, first, end;
    bool active;
};
NVFP4_DEVINL Part part_of(const Call &c, const Item &it, int t)
{
    Part p;
    p.token0 = it.token0 + t * c.tokens;
    p.active = p.token0 < it.len;
    int lo, hi, unused;
    key_range(c, it.len, p.token0, &lo, &unused);
    key_range(c, it.len, min(p.token0 + c.tokens, it.len) - 1, &unused, &hi);
    p.first = (lo - it.lo) / kTile;
    p.end = (hi - it.lo + kTile - 1) / kTile;
    return p;
}

// ---------------------------------------------------------------------------
// Load warp
// ---------------------------------------------------------------------------

// Items of a call in order: by place in the sequence (a sequence's last ones first), then by sequence, then by head.
struct Cursor {
    int level, chunk;  // place, and 32 sequences of which lane i holds the i-th
    int begin, len, places;  // the lane's: places of two row tiles
    uint32_t with;     // lanes whose sequence has the level's place
    int64_t pos;       // number of the first item of the level and chunk

    NVFP4_DEVINL void load(const Call &c, int lane, bool report)
    {
        const int b = chunk + lane;
        begin = len = 0;
        if (b < c.n_seqs) {
            len = c.total;
            if (c.offsets) {
                const int from = c.offsets[b], to = c.offsets[b + 1];
                const bool ok = from >= 0 && to >= from && to <= c.total;
                if (!ok && report)
                    kv::report_index(c.status, kStatusPromptOffsets);
                begin = from;
                len = ok ? to - from : 0;
            }
        }
        places = (len + 2 * c.tokens - 1) / (2 * c.tokens);
    }
    NVFP4_DEVINL void start(const Call &c, int lane)
    {
        level = 0;
        for (chunk = 0; chunk < c.n_seqs; chunk += 32) {
            load(c, lane, blockIdx.x == 0);
            level = max(level, places);
        }
        level = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)level) - 1;
        chunk = 0;
        pos = 0;
        if (c.n_seqs > 32)
            load(c, lane, false);
        with = __ballot_sync(0xFFFFFFFFu, places > level);
    }
    // Item number `want` (not before the last one asked for); false if there are not as many.
    NVFP4_DEVINL bool find(const Call &c, int lane, int64_t want, Item *it)
    {
        for (;;) {
            if (level < 0)
                return false;
            const int64_t count = (int64_t)__popc(with) * c.kv_heads;
            if (want < pos + count)
                break;
            pos += count;
            chunk += 32;
            if (chunk >= c.n_seqs) {
                chunk = 0;
                --level;
            }
            if (c.n_seqs > 32)
                load(c, lane, false);
            with = __ballot_sync(0xFFFFFFFFu, places > level);
        }
        const int k = (int)(want - pos), which = k / c.kv_heads;
        const int src = (int)__fns(with, 0, which + 1);
        it->begin = __shfl_sync(0xFFFFFFFFu, begin, src);
        it->len = __shfl_sync(0xFFFFFFFFu, len, src);
        it->token0 = level * 2 * c.tokens;
        it->head = k - which * c.kv_heads;
        const int last = min(it->token0 + 2 * c.tokens, it->len) - 1;
        key_range(c, it->len, it->token0, &it->lo, &it->all_hi);
        key_range(c, it->len, last, &it->all_lo, &it->hi);
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
    cur.start(c, lane);
    uint32_t ks = 0, vs = 0, qs[2] = {0, 0};  // loads so far
    const int64_t ctas = gridDim.x;
    bool ok = true;
    const auto load_k = [&](const Item &it, int tile) {
        const uint32_t slot = ks % C::kKs, round = ks / C::kKs;
        ++ks;
        if (round > 0 && !tc::mbar_wait(&sh->k_empty[slot], (round - 1) & 1))
            return false;
        const uint32_t bar = tc::smem_addr(&sh->k_full[slot]), at = smem + C::kKAt + slot * C::kOperand;
        tc::mbar_arrive_expect_tx_a(bar, C::kOperand);
        for (int b = 0; b < D / 64; ++b)
            tma_load_3d(at + b * kTile * 128, k_map, bar, 64 * b, it.head, it.begin + it.lo + tile * kTile);
        return true;
    };
    const auto load_v = [&](const Item &it, int tile) {
        const uint32_t slot = vs % C::kVs, round = vs / C::kVs;
        ++vs;
        if (round > 0 && !tc::mbar_wait(&sh->v_empty[slot], (round - 1) & 1))
            return false;
        const uint32_t bar = tc::smem_addr(&sh->v_full[slot]), at = smem + C::kVAt + slot * C::kOperand;
        tc::mbar_arrive_expect_tx_a(bar, C::kOperand);
        for (int b = 0; b < D / 64; ++b)
            tma_load_3d(at + b * kTile * 128, v_map, bar, 64 * b, it.head, it.begin + it.lo + tile * kTile);
        return true;
    };
    const auto load_q = [&](const Item &it, int t) {
        const uint32_t n = qs[t]++;
        if (n > 0 && !tc::mbar_wait(&sh->q_empty[t], (n - 1) & 1))
            return false;
        const uint32_t bar = tc::smem_addr(&sh->q_full[t]), at = smem + t * C::kOperand;
        tc::mbar_arrive_expect_tx_a(bar, c.group * c.tokens * D * 2);
        for (int b = 0; b < D / 64; ++b)
            tma_load_3d(at + b * kTile * 128, q_map, bar, 64 * b, it.head * c.group, it.begin + it.token0 + t * c.tokens);
        return true;
    };
    for (uint32_t n = 0;; ++n) {
        Item it;
        const bool any = cur.find(c, lane, n * ctas + (n & 1 ? ctas - 1 - blockIdx.x : blockIdx.x), &it);
        const uint32_t slot = n % kItems;
        if (lane == 0) {
            ok = n < kItems || tc::mbar_wait(&sh->item_empty[slot], (n / kItems - 1) & 1);
            if (!any)
                it.len = 0;
            sh->item[slot] = it;
            sh->bad[slot] = 0;
            tc::mbar_arrive(&sh->item_full[slot]);
            if (any && ok) {
                // the first keys do not wait for the queries before to be done with
                ok = load_k(it, 0) && load_q(it, 0) && (it.token0 + c.tokens >= it.len || load_q(it, 1)) && load_v(it, 0);
                for (int tile = 1; tile < it.tiles() && ok; ++tile)
                    ok = load_k(it, tile) && load_v(it, tile);
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!any || !ok)
            break;
    }
    // Nothing is in flight when the warp leaves: without a timeout the other warps have waited for every load.
    if (lane == 0 && !ok) {
        for (uint32_t i = ks > C::kKs ? ks - C::kKs : 0; i + 1 < ks; ++i)
            tc::mbar_wait(&sh->k_full[i % C::kKs], (i / C::kKs) & 1);
        for (uint32_t i = vs > C::kVs ? vs - C::kVs : 0; i + 1 < vs; ++i)
            tc::mbar_wait(&sh->v_full[i % C::kVs], (i / C::kVs) & 1);
    }
    return ok;
}

// ---------------------------------------------------------------------------
// MMA warp
// ---------------------------------------------------------------------------

// One thread issues every product, in the order
//     S0(0) S1(0)  then for each key tile i:  PV0(i) S0(i+1) PV1(i) S1(i+1),
// so that one row tile's products run while the other is in its softmax.  (With a thread for each row
// tile both came to wait for their softmax at the same time.)  Products of one thread run in
// the order of issue, which lets S(i+1) overwrite the scores that PV(i) reads as weights.
template <int D>
NVFP4_DEVINL bool mma_role(const Call &c, Shared *sh, uint32_t smem, uint32_t tmem)
{
    using C = Cfg<D>;
    constexpr uint32_t score_idesc = tc::idesc_f16kind(kTile, kTile, 1);
    constexpr uint32_t out_idesc = tc::idesc_f16kind(kTile, D, 1) | 1u << 16;  // B transposed
    uint32_t ks = 0, vs = 0, items[2] = {0, 0}, mine[2] = {0, 0};  // tiles of K and V so far, the row tiles' items and products P V
    bool ok = true;
    const auto score = [&](const Part &part, int t, int i) {
        const uint32_t k = smem + C::kKAt + (ks % C::kKs) * C::kOperand, q = smem + t * C::kOperand;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            const uint32_t at = (d / 4) * (kTile * 128) + (d % 4) * 32;
            const uint64_t base = 1ull << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
            tc::mma_bf16_ss(tmem + t * kTile, base | ((q + at) & 0x3FFFFu) >> 4, base | ((k + at) & 0x3FFFFu) >> 4, score_idesc,
                            d > 0);
        }
        tc::mma_commit(&sh->s_full[t]);
        if (i + 1 == part.end)
            tc::mma_commit(&sh->q_empty[t]);
    };
    const auto uses = [](const Part &part, int i) { return part.active && i >= part.first && i < part.end; };
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kItems;
        if (!(ok = tc::mbar_wait(&sh->item_full[slot], (n / kItems) & 1)))
            break;
        const Item it = sh->item[slot];
        tc::mbar_arrive(&sh->item_empty[slot]);
        if (it.len == 0)
            break;
        const Part part[2] = {part_of(c, it, 0), part_of(c, it, 1)};
        const int tiles = it.tiles();
        ok = tc::mbar_wait(&sh->k_full[ks % C::kKs], (ks / C::kKs) & 1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (part[t].active)
                ok = ok && tc::mbar_wait(&sh->q_full[t], items[t] & 1);
            if (ok && uses(part[t], 0))
                score(part[t], t, 0);
        }
        tc::mma_commit(&sh->k_empty[ks++ % C::kKs]);
        for (int i = 0; i < tiles && ok; ++i) {
            const uint32_t v_slot = vs % C::kVs, v_phase = (vs / C::kVs) & 1;
            const uint32_t v = smem + C::kVAt + v_slot * C::kOperand;
            ++vs;
            ok = tc::mbar_wait(&sh->v_full[v_slot], v_phase) && tc::mbar_wait(&sh->v_ready[v_slot], v_phase);
            const bool more = i + 1 < tiles;
            if (more)
                ok = ok && tc::mbar_wait(&sh->k_full[ks % C::kKs], (ks / C::kKs) & 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (uses(part[t], i)) {
                    // the item before has been read out
                    if (i == part[t].first && items[t] > 0)
                        ok = ok && tc::mbar_wait(&sh->o_free[t], (items[t] - 1) & 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && tc::mbar_wait(&sh->p_ready[t][h], mine[t] & 1);
                        if (!ok)
                            break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int j = 0; j < kTile / 32; ++j)
                            tc::mma_f16_ts(tmem + C::kOutCols + t * D, tmem + t * kTile + h * (kTile / 2) + 8 * j,
                                           desc_transposed(v + (h * (kTile / 32) + j) * 2048), out_idesc,
                                           i > part[t].first || h > 0 || j > 0);
                        if (h == 0)
                            tc::mma_commit(&sh->half_done[t]);
                    }
                    if (!ok)
                        break;
                    ++mine[t];
                    if (i + 1 == part[t].end)
                        tc::mma_commit(&sh->o_full[t]);
                }
                if (t == 1)
                    tc::mma_commit(&sh->v_empty[v_slot]);
                if (more && uses(part[t], i + 1))
                    score(part[t], t, i + 1);
            }
            if (more)
                tc::mma_commit(&sh->k_empty[ks++ % C::kKs]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
            items[t] += part[t].active;
    }
    // nothing of this thread's is in flight when it leaves
    tc::mma_commit(&sh->drain);
    return tc::mbar_wait(&sh->drain, 0) && ok;
}

// ---------------------------------------------------------------------------
// Scan warps
// ---------------------------------------------------------------------------

// All ones in the halves of a word of two bf16 that are infinities or NaN.
NVFP4_DEVINL uint32_t not_finite(uint32_t w)
{
    const uint32_t m = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    return (m >> 15) * 0xFFFFu;
}

template <int D>
NVFP4_DEVINL bool scan_role(const Call &c, Shared *sh, uint32_t smem, int warp, int lane)
{
    using C = Cfg<D>;
    uint32_t vs = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kItems;
        ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&sh->item_full[slot], (n / kItems) & 1));
        if (!ok)
            break;
        const Item it = sh->item[slot];
        const int tiles = it.len == 0 ? 0 : it.tiles();
        int mixed = 0;
        for (int i = 0; i < tiles; ++i, ++vs) {
            const uint32_t v_slot = vs % C::kVs;
            ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&sh->v_full[v_slot], (vs / C::kVs) & 1));
            if (!ok)
                break;
            if (it.mixed(i)) {
                // 32 rows of the tile, four at a time; 8 lanes to 128 bytes of a row
                const uint32_t at = smem + C::kVAt + v_slot * C::kOperand + warp * 32 * 128 + lane * 16;
                uint32_t bad = 0;
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const uint32_t a = at + b * kTile * 128 + r * 512;
                        const uint4 w = tc::lds128(a);
                        const uint4 m = make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w));
                        const bool any = (m.x | m.y | m.z | m.w) != 0;
                        const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, any);
                        if (lanes) {
                            if (any)
                                tc::sts128(a, make_uint4(w.x & ~m.x, w.y & ~m.y, w.z & ~m.z, w.w & ~m.w));
                            for (int k = 0; k < 4; ++k)
                                bad |= (lanes >> 8 * k & 0xFFu ? 1u : 0u) << (4 * r + k);
                        }
                    }
                }
                // keys that some row sees
                const int key0 = it.lo + i * kTile + warp * 32, some = it.hi - key0;
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
        }
        __syncwarp();
        if (lane == 0 && ok) {
            tc::mbar_arrive(&sh->scanned[slot]);
            tc::mbar_arrive(&sh->item_empty[slot]);
        }
        if (it.len == 0)
            break;
    }
    return ok;
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

template <int D>
NVFP4_DEVINL bool softmax_role(const Call &c, const uint16_t *v, int64_t v_ld, Shared *sh, uint32_t tmem, int tid)
{
    using C = Cfg<D>;
    const int t = tid / 128, r = tid % 128;  // row tile, and row of it: its lane of tensor memory
    const uint32_t lanes = (uint32_t)(r & ~31) << 16;
    const uint32_t scores = tmem + t * kTile + lanes, out = tmem + C::kOutCols + t * D + lanes;
    const int my_token = r / c.group, my_head = r - my_token * c.group;
    bool ok = true;
    uint32_t mine = 0, items = 0;  // the row tile's key tiles and items so far
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kItems;
        ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&sh->item_full[slot], (n / kItems) & 1));
        if (!ok)
            break;
        const Item it = sh->item[slot];
        if (it.len == 0)
            break;
        const Part part = part_of(c, it, t);
        if (!part.active) {
            __syncwarp();
            if (r % 32 == 0)
                tc::mbar_arrive(&sh->item_empty[slot]);
            continue;
        }
        const int token = part.token0 + my_token;
        const bool live = my_token < c.tokens && token < it.len;
        // rows beyond the last one: no key is masked, and none has any weight
        int lo = 0, hi = INT32_MAX;
        float top = 1e30f, f = 0.f;
        if (live) {
            key_range(c, it.len, token, &lo, &hi);
            top = -INFINITY;
            f = c.scale_log2;
        }
        float sum = 0.f;
        for (int i = part.first; i < part.end; ++i, ++mine) {
            const int key0 = it.lo + i * kTile;
            ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&sh->s_full[t], mine & 1));
            if (!ok)
                break;
            tc::fence_after_sync();
            const bool whole = __all_sync(0xFFFFFFFFu, key0 >= lo && key0 + kTile <= hi);
            const float g = whole ? f : 1.f;
            const uint64_t g2 = pack2(g, g);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // halves of the keys
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
                        const uint32_t see = range_bits(key0 + 64 * h + 32 * q, lo, hi);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            s[q][j] = see >> j & 1 ? __float_as_uint(__uint_as_float(s[q][j]) * f) : 0xFF800000u;  // -infinity
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
                                m = max3(m, __uint_as_float(s[q][j]) * g, __uint_as_float(s[q][j + 1]) * g);
                        }
                        const float next = over ? fmaxf(top, m - kHeadroom) : top;
                        // (nothing has been summed before the first reference)
                        const float shrink = top == next || top == -INFINITY ? 1.f : ex2(top - next);
                        top = next;
                        sum *= shrink;
                        const bool move = __any_sync(0xFFFFFFFFu, shrink != 1.f);
                        if (move && (i > part.first || h == 1)) {
                            // the first half's product may be under way (the tile before's is: these scores came after it)
                            if (h == 1)
                                ok = ok && tc::mbar_wait(&sh->half_done[t], mine & 1);
                            __syncwarp();
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
                    const float add = top == -INFINITY ? 0.f : -top;
                    const uint64_t add_2 = pack2(add, add);
                    uint64_t l2[2] = {0, 0};
                    uint32_t p[2][16];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 e = unpack2(fma2(
                                pack2(__uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1])), g2, add_2));
                            const float a = ex2(e.x), b = ex2(e.y);
                            l2[j & 1] = add2(l2[j & 1], pack2(a, b));
                            p[q][j] = f32x2_to_bf16x2(a, b);
                        }
                        tc::tmem_st_32x32b_x16(scores + 64 * h + 16 * q, p[q]);
                    }
                    const float2 la = unpack2(l2[0]), lb = unpack2(l2[1]);
                    l = (la.x + la.y) + (lb.x + lb.y);
                    over = l > kMostWeight;
                    if (!__any_sync(0xFFFFFFFFu, over))
                        break;
                }
                sum += l;
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (r % 32 == 0)
                    tc::mbar_arrive(&sh->p_ready[t][h]);
            }
        }
        ok = ok && tc::mbar_wait(&sh->o_full[t], items++ & 1) && tc::mbar_wait(&sh->scanned[slot], (n / kItems) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok)
            break;
        tc::fence_after_sync();
        const float inv = 1.f / sum;
        const bool bad = sh->bad[slot] != 0;
        const int64_t at = (int64_t)(it.begin + token) * c.out_ld + (int64_t)(it.head * c.group + my_head) * D;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
            uint32_t x[32];
            tc::tmem_ld_32x32b_x32(out + 32 * q, x);
            tc::tmem_ld_wait();
            settle(x);
            float o[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                o[j] = __uint_as_float(x[j]) * inv;
            if (bad && live) {
                // the infinities and NaN of V that the row sees in tiles from which they were taken out
                int mixed = 0;
#pragma unroll 1
                for (int i = 0; i < it.tiles(); ++i) {
                    if (!it.mixed(i))
                        continue;
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        const int key0 = it.lo + i * kTile + 32 * w;
                        uint32_t keys = sh->bad_keys[slot][mixed][w] & range_bits(key0, lo, hi);
                        for (; keys; keys &= keys - 1) {
                            const uint16_t *src = v + (int64_t)(it.begin + key0 + __ffs(keys) - 1) * v_ld + (int64_t)it.head * D + 32 * q;
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float e = __uint_as_float((uint32_t)src[j] << 16);
                                o[j] += isfinite(e) ? 0.f : e;
                            }
                        }
                    }
                    ++mixed;
                }
            }
            if (!live)
                continue;
            if (c.out_bf16) {
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.out) + at + 32 * q);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dst[j] = make_uint4(f32x2_to_bf16x2(o[8 * j], o[8 * j + 1]), f32x2_to_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                        f32x2_to_bf16x2(o[8 * j + 4], o[8 * j + 5]), f32x2_to_bf16x2(o[8 * j + 6], o[8 * j + 7]));
            } else {
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(c.out) + at + 32 * q);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (r % 32 == 0) {
            tc::mbar_arrive(&sh->o_free[t]);
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
            tc::mbar_init(&sh->half_done[t], 1);
            tc::mbar_init(&sh->o_full[t], 1);
            for (int h = 0; h < 2; ++h)
                tc::mbar_init(&sh->p_ready[t][h], 4);
        }
        tc::mbar_init(&sh->drain, 1);
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(&sh->item_full[i], 1);
            tc::mbar_init(&sh->item_empty[i], 1 + 8 + 4);  // MMA thread, softmax warps, scan warps
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
        ok = softmax_role<D>(c, v, v_ld, sh, tmem, tid);
        code = kTimeoutSoftmax;
    } else {
        give_regs<kOtherRegs>();
        if (warp == kLoadWarp) {
            ok = load_role<D>(c, &q_map, &k_map, &v_map, sh, smem, lane);
            code = kTimeoutLoad;
        } else if (warp == kMmaWarp) {
            if (elect_one()) {
                ok = mma_role<D>(c, sh, smem, tmem);
                code = kTimeoutMma;
            }
            __syncwarp();
        } else if (warp >= kScanWarp) {
            ok = scan_role<D>(c, sh, smem, warp - kScanWarp, lane);
            code = kTimeoutScan;
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
        (a->window > 0 && !a->causal) || !std::isfinite(a->scale) || (!a->offsets && a->n_seqs != 1))
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
    c.scale_log2 = args->scale * 1.4426950408889634f;
    int sms = 0;
    rc = current_num_sms(&sms);
    if (rc != NVFP4_OK)
        return rc;
    const cudaError_t e = args->head_dim == 64 ? prompt::launch<64>(*args, c, sms, (cudaStream_t)stream)
                                               : prompt::launch<128>(*args, c, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
