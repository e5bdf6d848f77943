// attention_plan.cuh -- how the attention kernels share a call's work out.
//
// An item is a block of query rows of one sequence and KV head: rows r of the
// sequence's new tokens times the query heads of one KV head (row r = token
// r / group, head r % group), RB at a time.  Its work is its key range in
// tiles of TK keys.  All items of all sequences form one list of tiles (heads
// fastest, then row blocks, then sequences), and CTA c of P takes the c-th of
// P equal ranges of it, whatever the lengths: long sequences are split over
// many CTAs, short ones share one, and every CTA has the same number of tiles
// to within one.  The lengths are on the device, so each CTA finds its range
// itself.  What an item costs beyond its tiles (its queries, joining the warps,
// a partial result) can be counted as tiles too: c.item_cost places without
// work stand before each item's tiles in the list.
//
// A CTA that holds a whole item writes its output rows.  Otherwise it leaves
// its partial result (accumulators, maximum and sum) in one of its two slots
// of the workspace (an item can reach into a CTA's range from the left or out
// of it to the right), and the last CTA of the item to arrive adds all partials
// in CTA order, so that the result does not depend on who was last.
#pragma once

#include "attention.h"
#include "attention_ops.cuh"

namespace nvfp4 {
namespace attn {

// 2^x, down to fp32's smallest numbers.
NVFP4_DEVINL float ex2_subnormal(float x)
{
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// s * 2^d for d <= 0 where 2^d may be too small for a float, but s * 2^d is not.
constexpr float kTwoSteps = -100.f;
NVFP4_DEVINL float times_pow2(float s, float d)
{
    const float half = ex2(0.5f * d);
    return s * half * half;
}

// Workspace: the status word (in the first 256 bytes), an arrival counter per
// CTA at byte 256, then two partial slots per CTA.
constexpr int kMaxCtas = 320;
constexpr size_t kCounterOffset = 256;
constexpr size_t kPartialOffset = kCounterOffset + kMaxCtas * sizeof(uint32_t);

// Rows of an item of the decode kernel, and the CTAs that it may have at most:
// two on an SM with one 8-row tile.  With two tiles 128 registers a thread do not
// hold the accumulators: one CTA of 255 took 23.6 us where two took 30.5 (one
// sequence of 30000 E4M3 keys, 16 rows).
constexpr int kMaxChunkCtas = kMaxCtas / 2;  // of the chunk kernel, one on an SM
constexpr int decode_block(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : 32; }
constexpr int decode_max_ctas(int block) { return block == 8 ? kMaxCtas : kMaxCtas / 2; }

struct Item {
    Seq seq;
    int b, rb, head;    // sequence, row block, KV head
    int row0, rows;     // rows of the block
    int lo, hi;         // keys that some row of the block may see
    int tile0, tiles;   // first tile (in units of TK keys from key 0) and their number
    int units;          // places in the list: the tiles, behind `c.item_cost` places without any
};

// Rows and key range of row block rb of an item's sequence.
template <int RB, int TK>
NVFP4_DEVINL void set_block(const Call &c, Item &it)
{
    it.row0 = it.rb * RB;
    it.rows = min(RB, it.seq.n * c.group - it.row0);
    int unused;
    key_range(c, it.seq, it.row0 / c.group, &it.lo, &unused);
    key_range(c, it.seq, (it.row0 + it.rows - 1) / c.group, &unused, &it.hi);
    it.tile0 = it.lo / TK;
    // an item without keys still has its zeros to write
    it.tiles = max(1, (it.hi + TK - 1) / TK - it.tile0);
    it.units = it.tiles + c.item_cost;
}

// Keys [lo, hi) that every row of an item sees.
NVFP4_DEVINL void common_keys(const Call &c, const Item &it, int *lo, int *hi)
{
    int unused;
    key_range(c, it.seq, it.row0 / c.group, &unused, hi);
    key_range(c, it.seq, (it.row0 + it.rows - 1) / c.group, lo, &unused);
    if (c.tree)
        *hi = min(*hi, max(it.seq.past, 0));
}

template <int RB>
NVFP4_DEVINL int row_blocks(const Call &c, const Seq &s) { return (s.n * c.group + RB - 1) / RB; }

struct Range {
    int64_t total;       // tiles of the call
    int64_t begin, end;  // of this CTA
    int ctas;            // that have a range
};

// (Lists of up to 2^22 tiles divide in 32 bits, which is several times faster.)
NVFP4_DEVINL int64_t range_start(int64_t total, int ctas, int cta)
{
    return total < (1 << 22) ? (int64_t)((uint32_t)total * (uint32_t)cta / (uint32_t)ctas) : total * cta / ctas;
}
// The CTA whose range holds tile u.
NVFP4_DEVINL int range_owner(int64_t total, int ctas, int64_t u)
{
    if (total < (1 << 22))
        return (int)((((uint32_t)u + 1) * (uint32_t)ctas + (uint32_t)total - 1) / (uint32_t)total) - 1;
    return (int)(((u + 1) * ctas + total - 1) / total) - 1;
}
static_assert(kMaxCtas < 1 << 9, "32-bit products of tiles and CTAs");

// Every thread of the CTA calls this: this CTA's range, its first item, and
// the list position of that item's first place.  `scratch`: shared memory,
// THREADS / 32 + 5 words of 64 bits.  Returns false if the CTA has no work.
//
// Row blocks are numbered as if every sequence had as many as the longest can
// have; thread t sums the t-th run of consecutive numbers (one long sequence
// is spread over the threads as well as many short ones), and a scan over the
// threads follows.
template <int RB, int TK, int THREADS>
__device__ bool find_range(const Call &c, int64_t *scratch, Range *range, Item *item, int64_t *item_begin)
{
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    // row blocks of a sequence (one at least, so that its lengths are looked at whatever max_q_len)
    const int most = max(1, (int)(((int64_t)c.max_q_len * c.group + RB - 1) / RB));
    const int64_t numbers = (int64_t)c.n_seqs * most;
    const int64_t per = numbers <= THREADS ? 1 : (numbers + THREADS - 1) / THREADS;
    const int64_t n0 = min(tid * per, numbers), n1 = min(n0 + per, numbers);
    // f(sequence and row block of each number of the run that is there, its tiles over all heads) until it returns true
    const auto each = [&](auto &&f) {
        if (n0 >= n1)
            return;
        Item it;
        it.b = most == 1 ? (int)n0 : (int)(n0 / most);
        it.rb = (int)(n0 - (int64_t)it.b * most);
        it.seq = load_seq(c, it.b);
        for (int64_t i = n0; i < n1; ++i) {
            if (it.rb < row_blocks<RB>(c, it.seq)) {
                set_block<RB, TK>(c, it);
                if (f(it, (int64_t)it.units * c.pool.heads))
                    return;
            }
            if (++it.rb == most && i + 1 < n1) {
                it.rb = 0;
                it.seq = load_seq(c, ++it.b);
            }
        }
    };
    int64_t mine = 0;
    each([&](const Item &, int64_t n) {
        mine += n;
        return false;
    });
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o)
            upto += v;
    }
    if (lane == 31)
        scratch[warp] = upto;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        const int64_t v = scratch[w];
        before += w < warp ? v : 0;
        total += v;
    }
    upto += before;
    range->total = total;
    range->ctas = (int)min((int64_t)gridDim.x, total);
    if ((int)blockIdx.x >= range->ctas)
        return false;
    range->begin = range_start(total, range->ctas, blockIdx.x);
    range->end = range_start(total, range->ctas, blockIdx.x + 1);
    if (range->begin >= upto - mine && range->begin < upto) {  // exactly one thread
        int64_t at = upto - mine;
        each([&](const Item &it, int64_t n) {
            if (range->begin >= at + n) {
                at += n;
                return false;
            }
            const int head = (int)((range->begin - at) / it.units);
            int64_t *out = scratch + THREADS / 32;
            out[0] = (int64_t)it.b << 32 | it.rb;
            out[1] = head;
            out[2] = at + (int64_t)head * it.units;
            out[3] = (int64_t)it.seq.q_begin << 32 | (uint32_t)it.seq.n;
            out[4] = (int64_t)it.seq.kv << 32 | (uint32_t)it.seq.past;
            return true;
        });
    }
    __syncthreads();
    const int64_t *out = scratch + THREADS / 32;
    item->b = (int)(out[0] >> 32);
    item->rb = (int)(out[0] & 0x7FFFFFFF);
    item->head = (int)out[1];
    *item_begin = out[2];
    item->seq = {(int)(out[3] >> 32), (int)out[3], (int)(out[4] >> 32), (int)out[4]};
    set_block<RB, TK>(c, *item);
    return true;
}

// The item after `item` in the list (there is one: the range has tiles left).
template <int RB, int TK>
NVFP4_DEVINL void next_item(const Call &c, Item *item)
{
    if (++item->head < c.pool.heads)
        return;
    item->head = 0;
    if (++item->rb >= row_blocks<RB>(c, item->seq)) {
        item->rb = 0;
        do
            item->seq = load_seq(c, ++item->b);
        while (item->seq.n == 0);
    }
    set_block<RB, TK>(c, *item);
}

}  // namespace attn
}  // namespace nvfp4
