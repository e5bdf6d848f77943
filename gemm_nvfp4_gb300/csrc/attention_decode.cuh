// attention_decode.cuh -- attention of few query rows per KV head (decode,
// speculative verify) over the quantised paged cache.
//
// With n new tokens and G query heads per KV head, each cached element is used
// by n * G rows: 2 n G multiply-adds a byte or so, far below what the tensor
// cores would need, so the kernel is bound by the cache's bytes, and at short
// contexts by the latency of its dependent steps.  What it does about that:
//
//  * one pass over the cache with a running maximum and sum per row;
//  * the key axis split over all SMs (attention_plan.cuh), because one decoded
//    sequence has only as many items as KV heads;
//  * every warp works alone on 16 keys at a time: it copies their codes, scales
//    and exponents into its own ring of shared memory with cp.async and no
//    barrier but its own, so 100 KB and more are in flight on an SM;
//  * codes turn into f16 fragments of the warp-level MMA in registers, exactly
//    (E4M3 and E2M1 * E4M3 have at most 6 significant bits), and never return to
//    memory.  mma.sync is enough: tcgen05 would want them in shared or tensor
//    memory, and fewer than 64 rows leave its 128-row tile mostly empty.
//
// The 16 x 8 score tile is S^T = K Q^T (keys x rows), and the output O^T = V^T P^T
// (elements x rows), so 8 rows, not 16, are the granule: NT tiles of 8.
// The contraction index of S is permuted so that a thread's K elements are
// consecutive bytes of a row, and so is the element index of O: the four keys
// (2t, 2t + 1, 2t + 8, 2t + 9) of thread column t and the D / 8 consecutive
// elements of thread row g give V^T fragments by byte interleaving alone.
//
// The row exponents never touch an element.  K's multiplies the score.  V's is
// added to the score's logarithm: with z = score + kv (in powers of two) the
// weight P = 2^(z - M) already carries V's magnitude, its largest values are near
// 2^7 whatever V's scale is, and f16 holds it to 2^-11; the softmax sum takes
// P * 2^-kv.  (Where V's exponents leave [-kNear, kNear), a key with most of the
// softmax and a tiny V could have a P of 0 beside a huge V of little weight: such
// a warp adds 2^(score - M) to its sum instead, and sums move to another M in two
// steps, since the factor alone may be 0.)  M trails the running maximum: it moves, and the accumulators are
// rescaled, only when some z exceeds it by 15 (P then stays below 2^15).
//
// f16 loses weights below 2^-32 of a row's largest.  That is far below what a bf16
// output shows, but not an fp32 one (where the large weights' V elements are
// zero, only the small ones are left).  For fp32 outputs (WIDE) V is turned
// into bf16 (also exact) and each weight into the sum of two bf16 numbers, with
// the exponent range of fp32 and 16 bits.
#pragma once

#include <cstdint>

#include "attention_plan.cuh"
#include "skinny.cuh"

namespace nvfp4 {
namespace attn {

namespace decode {

constexpr int kTile = 64;      // keys of a plan tile
constexpr int kStep = 16;      // keys of a warp step
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kHeadroom = 7.f, kSlack = 15.f;  // log2 of the largest P after and before a rescale
constexpr uint32_t kNear = 32;                   // P is far from 0 for what matters to the sum: 2 * 32 + 30 < 126
constexpr float kSumUnit = 0x1p-16f, kSumUnitLog2 = -16.f;  // the sum is kept in units of 2^16: P * 2^-kv reaches 2^115

template <int FMT, int D, int NT>
struct Cfg {
    using R = kv::Row<FMT, D>;
    static constexpr int kRows = 8 * NT;
    static constexpr int kCodeBytes = kStep * R::kCode, kScaleBytes = kStep * R::kScale;
    // stage: K codes, V codes, K scales, V scales, K exponents, V exponents
    static constexpr int kScaleAt = 2 * kCodeBytes, kExpAt = kScaleAt + 2 * kScaleBytes;
    static constexpr int kStageBytes = kExpAt + 2 * kStep;
    static constexpr int kCtasPerSm = NT == 1 ? 2 : 1;
    // the ring takes what shared memory is left beside Q and the tables
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kRowBytes = kRows * (4 + 4 + 4 + 8);  // score factor, key range, tree word
    static constexpr int kBudget = (kCtasPerSm == 2 ? 112 : 224) * 1024 - kQBytes - kRowBytes - 512;
    static constexpr int kFit = kBudget / (kWarps * kStageBytes);
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kOutStride = D + 2;  // floats; keeps the merge's writes on different banks
    static constexpr int kMergeBytes = kWarps * kRows * (kOutStride + 2) * 4;
    static constexpr int kJoinBytes = decode_max_ctas(kRows) * kRows * 2 * 4;  // statistics of all contributors
    static constexpr int kArena = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static_assert(kJoinBytes <= kArena, "join");
    static constexpr int kSmem = kArena + kQBytes + kRowBytes + 512;
    static constexpr int kSlotFloats = kRows * (D + 2);
    static_assert(kStages >= 2 && kSmem <= 227 * 1024, "shared memory");
};

NVFP4_DEVINL void cp_async16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
NVFP4_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
NVFP4_DEVINL void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

NVFP4_DEVINL void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

NVFP4_DEVINL uint32_t f32x2_to_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 x 8 transpose of 16-bit elements across the warp.
NVFP4_DEVINL uint32_t transpose_b16(uint32_t a)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

NVFP4_DEVINL uint32_t f32x2_to_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// An exponent byte less the first one that is near: below 2 kNear, a power of two, if
// it is, so that one comparison tells it of the bits of two.
NVFP4_DEVINL uint32_t from_near(uint32_t e) { return e - (127 - kNear); }
static_assert((kNear & (kNear - 1)) == 0, "one comparison for two bytes");

// Four E4M3 bytes to two f16x2.
NVFP4_DEVINL void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

NVFP4_DEVINL uint32_t lds8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// Words of `N` 32-bit values from shared memory, in the widest loads there are.
template <int N>
NVFP4_DEVINL void lds_words(uint32_t addr, uint32_t (&w)[N])
{
    if constexpr (N == 1) {
        w[0] = tc::lds32(addr);
    } else if constexpr (N == 2) {
        const uint2 v = tc::lds64(addr);
        w[0] = v.x, w[1] = v.y;
    } else {
        const uint4 v = tc::lds128(addr);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
}

// Byte address of 16-byte chunk `c` of row `r` among 16 rows of CPR chunks:
// rows fill 128-byte lines, and a line's chunks are permuted by an exclusive or
// that puts the chunks which the lanes of one load read on different banks
// (K: consecutive rows; V: every other row).
template <int CPR>
NVFP4_DEVINL uint32_t chunk_at(int r, int c)
{
    const int id = r * CPR + c, line = id >> 3;
    const int flip = CPR == 8 ? line & 7 : CPR == 4 ? 2 * (line & 3) : 2 * (line & 1);
    return line * 128 + ((id & 7) ^ flip) * 16;
}

// What a lane copies of every step: its chunks of codes (of K, and the same of
// V), and for the first lanes a chunk of scales or exponents.
struct LaneCopy {
    uint32_t code_at;  // of the first chunk in a stage; the others lie 512 bytes on (odd ones with bit 6 flipped, CPR = 8)
    uint32_t aux_at;   // in a stage; all ones: no scales or exponents for this lane
    uint32_t aux_from, aux_row;  // bytes from K's block of a page, and per row
};

template <int FMT, int D, int NT>
NVFP4_DEVINL LaneCopy lane_copy(const Call &c, int lane)
{
    using C = Cfg<FMT, D, NT>;
    using R = kv::Row<FMT, D>;
    constexpr int kChunks = R::kCode / 16, kScaleChunks = C::kScaleBytes / 16, per = kScaleChunks > 0 ? kScaleChunks : 1;
    const int shift = c.pool.page_shift;
    LaneCopy m;
    m.code_at = chunk_at<kChunks>(lane / kChunks, lane % kChunks);
    if (lane < 2 * kScaleChunks) {
        m.aux_at = C::kScaleAt + lane * 16;
        m.aux_from = lane / per * c.pool.block_bytes + (R::kCode << shift) + lane % per * 16;
        m.aux_row = R::kScale;
    } else if (lane < 2 * kScaleChunks + 2) {
        const int kv = lane - 2 * kScaleChunks;
        m.aux_at = C::kExpAt + kv * kStep;
        m.aux_from = kv * c.pool.block_bytes + ((R::kCode + R::kScale) << shift);
        m.aux_row = 1;
    } else {
        m.aux_at = ~0u;
        m.aux_from = m.aux_row = 0;
    }
    return m;
}

// A warp's copy of 16 keys from row `at` of a page (whose K block of the head is
// `blk`) into a stage of its ring.  `valid`: rows that hold keys; the others
// become zeros, so that nothing an unwritten slot holds can reach the second
// product.  (An exponent byte of 0, which no written row has, masks the key: so
// do keys whose page is not there.)
template <int FMT, int D, int NT>
NVFP4_DEVINL void load_step(const Call &c, const LaneCopy &m, const uint8_t *blk, int at, int valid, uint32_t stage,
                            int lane)
{
    using C = Cfg<FMT, D, NT>;
    using R = kv::Row<FMT, D>;
    constexpr int kChunks = R::kCode / 16, kMine = kStep * kChunks / 32;
    const uint8_t *const src = blk + at * R::kCode + lane * 16;
    const uint8_t *const aux = blk + m.aux_from + at * m.aux_row;
    const uint32_t even = stage + m.code_at, odd = stage + (kChunks == 8 ? m.code_at ^ 64 : m.code_at);
    if (valid == kStep) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t *const from = src + (kv ? c.pool.block_bytes : 0);
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((i & 1 ? odd : even) + kv * C::kCodeBytes + 512 * i),
                             "l"(from + 512 * i)
                             : "memory");
        }
        if (m.aux_at != ~0u)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(stage + m.aux_at), "l"(aux) : "memory");
    } else {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                cp_async16((i & 1 ? odd : even) + kv * C::kCodeBytes + 512 * i,
                           src + (kv ? c.pool.block_bytes : 0) + 512 * i, (i * 32 + lane) / kChunks < valid ? 16 : 0);
        }
        if (m.aux_at != ~0u) {
            // rows of this chunk that hold keys
            const int begin = m.aux_row == 1 ? 0 : lane % (C::kScaleBytes / 16 > 0 ? C::kScaleBytes / 16 : 1) * 16;
            cp_async16(stage + m.aux_at, aux, min(16, max(0, valid * (int)m.aux_row - begin)));
        }
    }
}

// K fragment words: thread (g, t) holds D / 4 consecutive elements of rows g
// and g + 8, and turns them into the A operands of D / 16 MMAs.
template <int FMT, int D, int NT, class F>
NVFP4_DEVINL void for_k_fragments(uint32_t stage, int g, int t, F &&f)
{
    using C = Cfg<FMT, D, NT>;
    using R = kv::Row<FMT, D>;
    constexpr int kBytes = R::kCode / 4, kChunks = R::kCode / 16;
    if constexpr (FMT == NVFP4_KV_E4M3) {
#pragma unroll
        for (int j = 0; j < kBytes / 16; ++j) {
            uint32_t a[4], b[4];
            lds_words(stage + chunk_at<kChunks>(g, t * (kBytes / 16) + j), a);
            lds_words(stage + chunk_at<kChunks>(g + 8, t * (kBytes / 16) + j), b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t r[4];
                e4m3x4_to_f16(a[i], r[0], r[2]);
                e4m3x4_to_f16(b[i], r[1], r[3]);
                f(j * 4 + i, r);
            }
        }
    } else {
        constexpr int kWords = kBytes / 4, kBlocks = D / 64;  // scale blocks of a thread's elements
        uint32_t a[kWords], b[kWords];
        lds_words(stage + chunk_at<kChunks>(g, t * kBytes / 16) + t * kBytes % 16, a);
        lds_words(stage + chunk_at<kChunks>(g + 8, t * kBytes / 16) + t * kBytes % 16, b);
        const uint32_t sa = stage + C::kScaleAt + g * R::kScale + t * kBlocks;
        uint32_t s2[kBlocks][2];
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t s = lds8(sa + h * 8 * R::kScale + j);
                s2[j][h] = e4m3x2_to_f16x2((uint16_t)(s * 0x101u));
            }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            uint32_t x[4], y[4];
            sk::e2m1x8_to_f16x2(a[w], x);
            sk::e2m1x8_to_f16x2(b[w], y);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t *s = s2[w / 2];
                const uint32_t r[4] = {sk::f16x2_mul(x[2 * i], s[0]), sk::f16x2_mul(y[2 * i], s[1]),
                                       sk::f16x2_mul(x[2 * i + 1], s[0]), sk::f16x2_mul(y[2 * i + 1], s[1])};
                f(w * 2 + i, r);
            }
        }
    }
}

// V fragments: thread (g, t) holds elements g * D/8 .. of keys 2t, 2t + 1,
// 2t + 8, 2t + 9; MMA tile i covers elements 2i and 2i + 1 of each thread row.
// f16 operands are the codes' values (times block scales); WIDE: bf16 operands,
// the same times kWideUnit.
template <int FMT>
constexpr float kWideUnit = FMT == NVFP4_KV_E4M3 ? 0x1p-120f : 0x1p-9f;

// Two E4M3 bytes at bits 8..15 and 24..31 to bf16x2 holding e4m3 * 2^-120 each:
// sign to the sign, exponent and fraction fields to the low end of bf16's
// exponent and the high end of its fraction; E4M3's subnormals land on bf16's.
NVFP4_DEVINL uint32_t e4m3x2_to_bf16x2(uint32_t r) { return (r & 0x80008000u) | ((r >> 4) & 0x07F007F0u); }

// E2M1 codes at bits 4 N .. of both halves to bf16x2, times `mult`: the bits
// placed as above read e2m1 * 2^-126, and mult = scale * 2^117.
template <int N>
NVFP4_DEVINL uint32_t e2m1x2_to_bf16x2(uint32_t x, uint32_t mult)
{
    const uint32_t mag = N == 0 ? x << 6 : N == 1 ? x << 2 : N == 2 ? x >> 2 : x >> 6;
    const uint32_t sign = N == 0 ? x << 12 : N == 1 ? x << 8 : N == 2 ? x << 4 : x;
    return bf16x2_mul((mag & 0x01C001C0u) | (sign & 0x80008000u), mult);
}

// Takes the bytes that are not a number (no append writes them, but a slot that
// none has written may hold them) out of a step's V codes or block scales: a weight
// of zero does not keep such a key away from the rows that do not see it.  Steps
// whose keys every row sees need none of this.
template <int FMT, int D, int NT>
NVFP4_DEVINL void clear_nan_codes(uint32_t stage, int lane)
{
    using C = Cfg<FMT, D, NT>;
    if constexpr (FMT == NVFP4_KV_E4M3) {
#pragma unroll 1
        for (int i = 0; i < C::kCodeBytes / 512; ++i) {
            const uint32_t at = stage + C::kCodeBytes + i * 512 + lane * 16;
            const uint4 w = tc::lds128(at);
            tc::sts128(at, make_uint4(kv::without_nan(w.x), kv::without_nan(w.y), kv::without_nan(w.z), kv::without_nan(w.w)));
        }
    } else if (lane < C::kScaleBytes / 4) {
        const uint32_t at = stage + C::kScaleAt + C::kScaleBytes + lane * 4;
        tc::sts32(at, kv::without_nan(tc::lds32(at)));
    }
    __syncwarp();
}

template <int FMT, int D, int NT, bool WIDE, class F>
NVFP4_DEVINL void for_v_fragments(uint32_t stage, int g, int t, F &&f)
{
    using C = Cfg<FMT, D, NT>;
    using R = kv::Row<FMT, D>;
    constexpr int kBytes = R::kCode / 8, kChunks = R::kCode / 16, kWords = kBytes / 4;
    uint32_t w[4][kWords];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const int r = 2 * t + (h & 1) + (h >> 1) * 8;
        lds_words(stage + C::kCodeBytes + chunk_at<kChunks>(r, g * kBytes / 16) + g * kBytes % 16, w[h]);
    }
    if constexpr (FMT == NVFP4_KV_E4M3) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t r[4];
                if constexpr (WIDE) {
                    const uint32_t even = half ? 0x6020 : 0x4000, odd = half ? 0x7030 : 0x5010;
                    r[0] = e4m3x2_to_bf16x2(prmt(w[0][j], w[1][j], even));
                    r[1] = e4m3x2_to_bf16x2(prmt(w[0][j], w[1][j], odd));
                    r[2] = e4m3x2_to_bf16x2(prmt(w[2][j], w[3][j], even));
                    r[3] = e4m3x2_to_bf16x2(prmt(w[2][j], w[3][j], odd));
                } else {
                    // bytes (key 2t, key 2t + 1) of two consecutive elements
                    const uint32_t sel = half ? 0x7362 : 0x5140;
                    e4m3x4_to_f16(prmt(w[0][j], w[1][j], sel), r[0], r[1]);
                    e4m3x4_to_f16(prmt(w[2][j], w[3][j], sel), r[2], r[3]);
                }
                f(2 * j + half, r);
            }
        }
    } else {
        uint32_t s2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t sa = stage + C::kScaleAt + C::kScaleBytes + (2 * t + h * 8) * R::kScale + g * (D / 8) / 16;
            if constexpr (WIDE)
                s2[h] = f32x2_to_bf16x2(e4m3_to_f32(lds8(sa)) * 0x1p117f, e4m3_to_f32(lds8(sa + R::kScale)) * 0x1p117f);
            else
                s2[h] = e4m3x2_to_f16x2((uint16_t)(lds8(sa) | lds8(sa + R::kScale) << 8));
        }
        constexpr uint32_t m = 0x0F0F0F0Fu;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            if constexpr (WIDE) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x7632 : 0x5410;  // four elements of key 2t, then of key 2t + 1
                    const uint32_t x = prmt(w[0][j], w[1][j], sel), y = prmt(w[2][j], w[3][j], sel);
                    const uint32_t r0[4] = {e2m1x2_to_bf16x2<0>(x, s2[0]), e2m1x2_to_bf16x2<1>(x, s2[0]),
                                            e2m1x2_to_bf16x2<0>(y, s2[1]), e2m1x2_to_bf16x2<1>(y, s2[1])};
                    f(4 * j + 2 * half, r0);
                    const uint32_t r1[4] = {e2m1x2_to_bf16x2<2>(x, s2[0]), e2m1x2_to_bf16x2<3>(x, s2[0]),
                                            e2m1x2_to_bf16x2<2>(y, s2[1]), e2m1x2_to_bf16x2<3>(y, s2[1])};
                    f(4 * j + 2 * half + 1, r1);
                }
            } else {
                // nibbles (key 2t low, key 2t + 1 high) of the even elements, then of the odd ones
                uint32_t e0[4], o0[4], e1[4], o1[4];
                sk::e2m1x8_to_f16x2((w[0][j] & m) | ((w[1][j] << 4) & ~m), e0);
                sk::e2m1x8_to_f16x2(((w[0][j] >> 4) & m) | (w[1][j] & ~m), o0);
                sk::e2m1x8_to_f16x2((w[2][j] & m) | ((w[3][j] << 4) & ~m), e1);
                sk::e2m1x8_to_f16x2(((w[2][j] >> 4) & m) | (w[3][j] & ~m), o1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t r[4] = {sk::f16x2_mul(e0[i], s2[0]), sk::f16x2_mul(o0[i], s2[0]),
                                           sk::f16x2_mul(e1[i], s2[1]), sk::f16x2_mul(o1[i], s2[1])};
                    f(4 * j + i, r);
                }
            }
        }
    }
}

template <int FMT, int D, int NT, bool WIDE>
__global__ void __launch_bounds__(kThreads, Cfg<FMT, D, NT>::kCtasPerSm) decode_kernel(Call c, uint8_t *workspace)
{
    // WIDE: bf16 weights enter times kLift (which keeps E4M3's products, at kWideUnit, in fp32's range)
    constexpr float kLift = FMT == NVFP4_KV_E4M3 ? 0x1p100f : 1.f;
    constexpr float kOutUnit = WIDE ? kSumUnit / (kLift * kWideUnit<FMT>) : kSumUnit;
    using C = Cfg<FMT, D, NT>;
    constexpr int KS = D / 16;      // MMAs along D
    constexpr bool kQInRegs = NT == 1;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *const q_smem = smem + C::kArena;
    float *const q_factor = reinterpret_cast<float *>(q_smem + C::kQBytes);
    int *const q_lo = reinterpret_cast<int *>(q_factor + C::kRows), *const q_hi = q_lo + C::kRows;
    uint64_t *const q_tree = reinterpret_cast<uint64_t *>(q_hi + C::kRows);
    int64_t *const scratch = reinterpret_cast<int64_t *>(q_tree + C::kRows);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;

    tc::griddep_launch_dependents();
    tc::griddep_wait();
    Range range;
    Item it;
    int64_t item_begin;
    if (!find_range<C::kRows, kTile, kThreads>(c, scratch, &range, &it, &item_begin))
        return;
    const uint32_t ring = tc::smem_addr(smem) + warp * C::kStages * C::kStageBytes;
    const int page_mask = (1 << c.pool.page_shift) - 1;
    const LaneCopy copy = lane_copy<FMT, D, NT>(c, lane);
    uint32_t *const counters = reinterpret_cast<uint32_t *>(workspace + kCounterOffset);
    float *const partials = reinterpret_cast<float *>(workspace + kPartialOffset);

    for (int64_t u = range.begin; u < range.end;) {
        const int64_t tiles_begin = item_begin + c.item_cost, item_end = item_begin + it.units;
        const int64_t seg_end = min(item_end, range.end);
        if (seg_end <= tiles_begin) {  // no tile of the item is this CTA's
            u = seg_end;
            if (u < range.end) {
                item_begin = item_end;
                next_item<C::kRows, kTile>(c, &it);
            }
            continue;
        }
        u = max(u, tiles_begin);
        const int key0 = (it.tile0 + (int)(u - tiles_begin)) * kTile;
        const int steps = (int)(seg_end - u) * (kTile / kStep);
        const int mine = (steps - warp + kWarps - 1) / kWarps;  // steps of this warp: warp, warp + kWarps, ...
        const int32_t *const table = c.table + (int64_t)it.b * c.table_width;

        // Copies run kStages - 1 steps ahead; page numbers one step ahead of the copies.
        const uint8_t *const head_blk = kv::block_ptr(c.pool, 0, it.head, 0);
        int next_key = key0 + warp * kStep, next_left = mine;  // of the step whose page is looked up next
        uint32_t next_stage = ring;
        const auto page_at = [&](int key) {
            return next_left > 0 && key < it.hi && key + kStep > it.lo ? table[key >> c.pool.page_shift] : -1;
        };
        int page_next = page_at(next_key);
        const auto issue = [&] {
            const int page = page_next, key = next_key;
            const bool any = next_left > 0;
            next_key += kWarps * kStep;
            --next_left;
            page_next = page_at(next_key);
            if (any) {
                const bool used = key < it.hi && key + kStep > it.lo;
                int valid = used ? min(kStep, it.seq.kv - key) : 0;
                if (used && (page < 0 || page >= c.pool.n_pages)) {
                    kv::report_index(c.pool.status, kStatusKvAttention);
                    valid = 0;
                }
                const uint8_t *blk = head_blk + (valid > 0 ? (int64_t)((uint64_t)(uint32_t)page * (uint32_t)c.pool.page_bytes) : 0);
                load_step<FMT, D, NT>(c, copy, blk, key & page_mask, valid, next_stage, lane);
                next_stage = next_stage == ring + (C::kStages - 1) * C::kStageBytes ? ring : next_stage + C::kStageBytes;
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i)
            issue();

        // Q rows to f16 fragments (scaled by a power of two), their score factors and key ranges
        for (int r = warp; r < C::kRows; r += kWarps) {
            uint2 x = make_uint2(0, 0);
            int64_t row = 0;
            if (r < it.rows) {
                const int tok = (it.row0 + r) / c.group, hq = it.head * c.group + (it.row0 + r) % c.group;
                row = it.seq.q_begin + tok;
                if (lane < D / 4)
                    x = *reinterpret_cast<const uint2 *>(c.q + row * c.q_ld + (int64_t)hq * D + lane * 4);
                if (lane == 0) {
                    int lo, hi;
                    key_range(c, it.seq, tok, &lo, &hi);
                    q_lo[r] = lo;
                    q_hi[r] = hi;
                    q_tree[r] = c.tree ? c.tree[row] : 0;
                }
            } else if (lane == 0) {
                q_lo[r] = q_hi[r] = 0;
                q_tree[r] = 0;
            }
            const uint32_t m2 = __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
            const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
            const int e = max((int)(m >> 7), 15);  // exponent field of the largest; 255: not a number
            const float up = e == 255 ? NAN : __uint_as_float((uint32_t)(268 - e) << 23);
            if (lane < D / 4) {
                uint2 h;
                h.x = f32x2_to_f16x2(__uint_as_float(x.x << 16) * up, __uint_as_float(x.x & 0xFFFF0000u) * up);
                h.y = f32x2_to_f16x2(__uint_as_float(x.y << 16) * up, __uint_as_float(x.y & 0xFFFF0000u) * up);
                // element 4 * lane belongs to thread column lane / KS, MMA lane % KS, of row r
                const int at = ((r / 8 * KS + lane % KS) * 32 + r % 8 * 4 + lane / KS) * 8;
                *reinterpret_cast<uint2 *>(q_smem + at) = h;
            }
            if (lane == 0)
                q_factor[r] = c.scale_log2 * __uint_as_float((uint32_t)max(e - 14, 1) << 23);
        }
        __syncthreads();

        uint2 qf[kQInRegs ? KS : 1];
        const uint32_t q_addr = tc::smem_addr(q_smem) + lane * 8;
        if constexpr (kQInRegs) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
                qf[i] = tc::lds64(q_addr + i * 256);
        }
        float factor[NT][2];
        int lo_last, hi_first;  // keys from lo_last to hi_first are seen by every row
        common_keys(c, it, &lo_last, &hi_first);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            factor[n][0] = q_factor[n * 8 + 2 * t];
            factor[n][1] = q_factor[n * 8 + 2 * t + 1];
        }

        float top[NT][2], sum[NT][2], o[NT][KS][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            top[n][0] = top[n][1] = -INFINITY;
            sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
                o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        }

        float limit[NT][2], base[NT][2];  // top + kSlack, and top or 0 where there is none yet
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            limit[n][0] = limit[n][1] = -INFINITY;
            base[n][0] = base[n][1] = 0.f;
        }
        int key = key0 + warp * kStep;
        uint32_t stage = ring;
        bool far = false;  // the warp has met a V exponent beyond kNear
        for (int i = 0; i < mine; ++i, key += kWarps * kStep) {
            cp_async_wait<C::kStages - 2>();
            __syncwarp();
            issue();

            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            for_k_fragments<FMT, D, NT>(stage, g, t, [&](int k, const uint32_t (&a)[4]) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint2 b = kQInRegs ? qf[kQInRegs ? k : 0] : tc::lds64(q_addr + (n * KS + k) * 256);
                    mma_f16_16816(s[n], a, b.x, b.y);
                }
            });

            // exponents of keys g and g + 8
            float z[NT][4], unscale[2];
            bool over;
            {
                const uint32_t ea = stage + C::kExpAt + g;
                // K's mark of a row that is not a number reads infinity here, and its codes are zeros: NaN again
                const float fk[2] = {__uint_as_float(lds8(ea) << 23), __uint_as_float(lds8(ea + 8) << 23)};
                const uint32_t ev[2] = {lds8(ea + kStep), lds8(ea + kStep + 8)};
                float kv[2];
                over = (from_near(ev[0]) | from_near(ev[1])) >= 2 * kNear;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the byte as a float: 2^23 + ev - (2^23 + 127)
                    kv[h] = __uint_as_float(0x4B000000u | ev[h]) - 8388735.f;
                    kv[h] = ev[h] == kv::kNanRow ? NAN : ev[h] == 0 ? -INFINITY : kv[h];
                    // finite for a NaN row too: masked, its weight of 0 must add 0
                    unscale[h] = __uint_as_float((uint32_t)max(254 - (int)ev[h], 0) << 23) * kSumUnit;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        z[n][h] = fmaf(s[n][h] * factor[n][h & 1], fk[h >> 1], kv[h >> 1]);
                }
            }
            if (key < lo_last || key + kStep > hi_first) {
                if (key < lo_last || min(key + kStep, it.seq.kv) > hi_first)
                    clear_nan_codes<FMT, D, NT>(stage, lane);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int r = n * 8 + 2 * t + (h & 1), j = key + g + (h >> 1) * 8;
                        bool see = j >= q_lo[r] && j < q_hi[r];
                        if (c.tree && j >= it.seq.past)
                            see &= j - it.seq.past < 64 && (q_tree[r] >> ((j - it.seq.past) & 63) & 1);
                        z[n][h] = see ? z[n][h] : -INFINITY;
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    over |= z[n][h] > limit[n][h & 1];
            }
            if (__any_sync(0xFFFFFFFFu, over)) {
                const uint32_t e0 = lds8(stage + C::kExpAt + kStep + g), e1 = lds8(stage + C::kExpAt + kStep + g + 8);
                far |= __any_sync(0xFFFFFFFFu, (from_near(e0) >= 2 * kNear && e0 != 0) || (from_near(e1) >= 2 * kNear && e1 != 0));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float m = fmaxf(z[n][h], z[n][h + 2]);
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                        const float next = fmaxf(top[n][h], m - kHeadroom);
                        const float shrink = next == -INFINITY ? 1.f : ex2(top[n][h] - next);
                        limit[n][h] = next + kSlack;
                        base[n][h] = next == -INFINITY ? 0.f : next;
                        sum[n][h] = far && next != -INFINITY ? times_pow2(sum[n][h], top[n][h] - next) : sum[n][h] * shrink;
                        top[n][h] = next;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[n][k][h] *= shrink;
                            o[n][k][h + 2] *= shrink;
                        }
                    }
                }
            }
            if (far) {  // these keys' shares as they are, not from their weights
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // finite, whatever the row
                    const float kv = __uint_as_float(0x4B000000u | lds8(stage + C::kExpAt + kStep + g + 8 * h)) - 8388735.f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        sum[n][0] += ex2_subnormal(z[n][2 * h] - (base[n][0] + kv - kSumUnitLog2));
                        sum[n][1] += ex2_subnormal(z[n][2 * h + 1] - (base[n][1] + kv - kSumUnitLog2));
                    }
                }
            }
            uint32_t p[NT][WIDE ? 4 : 2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float w[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    w[h] = ex2(z[n][h] - base[n][h & 1]);
                    if (!far)
                        sum[n][h & 1] = fmaf(w[h], unscale[h >> 1], sum[n][h & 1]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (WIDE) {
                        const float a = w[2 * h] * kLift, b = w[2 * h + 1] * kLift;
                        const uint32_t hi = f32x2_to_bf16x2(a, b);
                        p[n][h] = transpose_b16(hi);
                        p[n][h + 2] = transpose_b16(
                            f32x2_to_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u)));
                    } else {
                        p[n][h] = transpose_b16(f32x2_to_f16x2(w[2 * h], w[2 * h + 1]));
                    }
                }
            }
            for_v_fragments<FMT, D, NT, WIDE>(stage, g, t, [&](int k, const uint32_t (&a)[4]) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (WIDE) {
                        mma_bf16_16816(o[n][k], a, p[n][2], p[n][3]);
                        mma_bf16_16816(o[n][k], a, p[n][0], p[n][1]);
                    } else {
                        mma_f16_16816(o[n][k], a, p[n][0], p[n][1]);
                    }
                }
            });
            stage = stage == ring + (C::kStages - 1) * C::kStageBytes ? ring : stage + C::kStageBytes;
        }
        cp_async_wait<0>();
        __syncthreads();  // every warp is done with its ring: the arena now holds the warps' results

        float *const merge = reinterpret_cast<float *>(smem);
        float *const stats = merge + kWarps * C::kRows * C::kOutStride;  // [warp][row] top, then sum
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = sum[n][h];
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
                const int r = n * 8 + 2 * t + h;
                if (g == 0) {
                    stats[warp * C::kRows + r] = top[n][h];
                    stats[(kWarps + warp) * C::kRows + r] = x;
                }
                float *dst = merge + (warp * C::kRows + r) * C::kOutStride + g * (D / 8);
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    *reinterpret_cast<float2 *>(dst + 2 * k) = make_float2(o[n][k][h], o[n][k][h + 2]);
            }
        }
        __syncthreads();

        const bool whole = u == tiles_begin && seg_end == item_end;
        // sums of the CTA: thread handles element pairs of rows; `emit` gets (row, element, values, top, sum)
        const auto merged = [&](auto &&emit) {
            for (int x = tid; x < it.rows * (D / 2); x += kThreads) {
                const int r = x / (D / 2), d = x % (D / 2) * 2;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    m = fmaxf(m, stats[w * C::kRows + r]);
                float2 acc = make_float2(0.f, 0.f);
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float tw = stats[w * C::kRows + r];
                    const float f = tw == -INFINITY ? 0.f : ex2(tw - m);  // 0 * NaN stays NaN
                    const float2 v = *reinterpret_cast<const float2 *>(merge + (w * C::kRows + r) * C::kOutStride + d);
                    acc.x = fmaf(f, v.x, acc.x);
                    acc.y = fmaf(f, v.y, acc.y);
                    const float s = stats[(kWarps + w) * C::kRows + r];
                    l = tw - m < kTwoSteps ? l + times_pow2(s, tw - m) : fmaf(f, s, l);
                }
                emit(r, d, acc, m, l);
            }
        };
        const auto store = [&](int r, int d, float2 acc, float l) {
            const float inv = l == 0.f ? 0.f : kOutUnit / l;
            const int tok = (it.row0 + r) / c.group, hq = it.head * c.group + (it.row0 + r) % c.group;
            const int64_t at = (int64_t)(it.seq.q_begin + tok) * c.out_ld + (int64_t)hq * D + d;
            if (c.out_bf16) {
                uint32_t v;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(acc.y * inv), "f"(acc.x * inv));
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(c.out) + at) = v;
            } else {
                *reinterpret_cast<float2 *>(static_cast<float *>(c.out) + at) = make_float2(acc.x * inv, acc.y * inv);
            }
        };
        if (whole) {
            merged([&](int r, int d, float2 acc, float, float l) { store(r, d, acc, l); });
        } else {
            const int first = range_owner(range.total, range.ctas, tiles_begin);
            const int last = range_owner(range.total, range.ctas, item_end - 1);
            float *slot = partials + ((int64_t)blockIdx.x * 2 + ((int)blockIdx.x == first ? 1 : 0)) * C::kSlotFloats;
            merged([&](int r, int d, float2 acc, float m, float l) {
                *reinterpret_cast<float2 *>(slot + r * D + d) = acc;
                if (d == 0)
                    *reinterpret_cast<float2 *>(slot + C::kRows * D + r * 2) = make_float2(m, l);
            });
            __syncthreads();  // before the release below: it covers every thread's stores
            if (tid == 0) {
                uint32_t seen;
                asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(seen) : "l"(counters + first) : "memory");
                const bool done = seen == (uint32_t)(last - first);
                if (done)
                    counters[first] = 0;
                scratch[0] = done;
            }
            __syncthreads();
            if (scratch[0]) {
                // the first contributor holds the item from its begin on (slot 1), the others have it from the left
                const int n = last - first + 1;
                const float *const from = partials + (int64_t)first * 2 * C::kSlotFloats;
                const auto slot_of = [&](int i) { return from + (int64_t)(i == 0 ? 1 : 2 * i) * C::kSlotFloats; };
                float *const weight = merge;  // [contributor][row]: top, then 2^(top - largest)
                for (int x = tid; x < n * C::kRows; x += kThreads) {
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(slot_of(x / C::kRows) + C::kRows * D +
                                                                              x % C::kRows * 2));
                    weight[x] = ml.x;
                    weight[n * C::kRows + x] = ml.y;
                }
                __syncthreads();
                for (int r = warp; r < it.rows; r += kWarps) {
                    float m = -INFINITY;
                    for (int i = lane; i < n; i += 32)
                        m = fmaxf(m, weight[i * C::kRows + r]);
#pragma unroll
                    for (int o2 = 16; o2 > 0; o2 /= 2)
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o2));
                    for (int i = lane; i < n; i += 32) {
                        const float tw = weight[i * C::kRows + r];
                        weight[i * C::kRows + r] = tw == -INFINITY ? 0.f : ex2(tw - m);
                        // a sum (none is negative) that has been brought to m already: with its sign turned
                        if (tw - m < kTwoSteps)
                            weight[(n + i) * C::kRows + r] = -times_pow2(weight[(n + i) * C::kRows + r], tw - m);
                    }
                }
                __syncthreads();
                for (int x = tid; x < it.rows * (D / 4); x += kThreads) {
                    const int r = x / (D / 4), d = x % (D / 4) * 4;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    float l = 0.f;
#pragma unroll 8
                    for (int i = 0; i < n; ++i) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(slot_of(i) + r * D + d));
                        const float f = weight[i * C::kRows + r];
                        acc.x = fmaf(f, v.x, acc.x);
                        acc.y = fmaf(f, v.y, acc.y);
                        acc.z = fmaf(f, v.z, acc.z);
                        acc.w = fmaf(f, v.w, acc.w);
                        const float s = weight[(n + i) * C::kRows + r];
                        l = s < 0.f ? l - s : fmaf(f, s, l);
                    }
                    store(r, d, make_float2(acc.x, acc.y), l);
                    store(r, d + 2, make_float2(acc.z, acc.w), l);
                }
            }
        }
        u = seg_end;
        if (u < range.end) {
            item_begin = item_end;
            next_item<C::kRows, kTile>(c, &it);
            __syncthreads();  // the arena and the row tables are free again
        }
    }
}

template <int FMT, int D, int NT, bool WIDE>
cudaError_t launch(const Call &c, uint8_t *workspace, int num_sms, cudaStream_t stream)
{
    using C = Cfg<FMT, D, NT>;
    static std::once_flag once[kMaxDevices];
    static cudaError_t results[kMaxDevices];
    const auto kernel = decode_kernel<FMT, D, NT, WIDE>;
    Call call = c;
    // An item costs a CTA about as much as four to six of its tiles.  E4M3, 8 KV heads: 64 sequences of 258 to 8192
    // keys 61.9 us at 3, 59.7 at 4, 58.9 to 59.7 at 6, 59.6 at 9; 32 x 2000 with 24 rows 56.6 at 4, 55.9 at 6.
    // Sequences x cached tokens, at 0 and 4: 4 x 4000 with 4 rows 15.8 and 13.3 us, 8 x 4000 20.5 and 18.9,
    // 8 x 300 with 24 rows 23.5 and 14.6; slower is 12 x 1000 with 24 rows, 24.7 and 26.9.  With 8 items it
    // takes CTAs from the tiles: 1 x 1000 with 24 rows 14.0 and 17.8.
    const int64_t items = (int64_t)c.n_seqs * c.pool.heads;
    call.item_cost = items >= 128 ? 6 : items >= 32 ? 4 : 0;
    const cudaError_t e = once_per_device(once, results, [kernel] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess)
        return e;
    constexpr int most = decode_max_ctas(C::kRows);
    const int grid = num_sms * C::kCtasPerSm;
    return launch_dependent(kernel, dim3(grid < most ? grid : most), kThreads, C::kSmem, stream, call, workspace);
}

template <int FMT, int D, bool WIDE>
cudaError_t launch_rows(const Call &c, uint8_t *workspace, int num_sms, cudaStream_t stream)
{
    // the fewest 8-row tiles that hold a sequence's rows: tiles without rows cost as much as full ones
    const int64_t rows = (int64_t)c.max_q_len * c.group;
    const int block = decode_block(rows);
    if constexpr (WIDE) {  // (bf16 calls of more than 24 rows go to the chunk kernel)
        if (block == 32)
            return launch<FMT, D, 4, WIDE>(c, workspace, num_sms, stream);
    }
    return block == 8    ? launch<FMT, D, 1, WIDE>(c, workspace, num_sms, stream)
           : block == 16 ? launch<FMT, D, 2, WIDE>(c, workspace, num_sms, stream)
                         : launch<FMT, D, 3, WIDE>(c, workspace, num_sms, stream);
}

template <int FMT>
cudaError_t launch_format(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (c.out_bf16)
        return head_dim == 64 ? launch_rows<FMT, 64, false>(c, ws, num_sms, stream)
                              : launch_rows<FMT, 128, false>(c, ws, num_sms, stream);
    return head_dim == 64 ? launch_rows<FMT, 64, true>(c, ws, num_sms, stream)
                          : launch_rows<FMT, 128, true>(c, ws, num_sms, stream);
}

}  // namespace decode
}  // namespace attn
}  // namespace nvfp4
