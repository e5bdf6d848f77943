// rope.cu -- rotary positions with one position per axis and token (nvfp4_rope;
// include/nvfp4.h has the definition).
//
// An angle is position * frequency, and only its fraction of a turn counts.  In fp32
// that product is off by 0.06 radians at position 2^20; here a frequency is a 64-bit
// fixed-point fraction of a turn, made once on the host, and the product of the two
// integers modulo 2^64 is the angle's fraction with an error of |position| * 2^-65
// turns, for the price of one integer multiplication.
//
// Memory bounds it: every element is read and written once, the cosines and sines are shared by all heads of a token.
// Measured on one GB300: 8192 tokens of 40 and 8 bf16 heads of 128, three axes (202 MB) 31.7 us, 6.4 TB/s, 0.94 of the
// measured copy rate (63 us an element at a time, 48 us with a token's loads behind its cosines and sines); 4999 tokens of 16 and 16
// fp32 heads of 64, half of each turned in neighbouring pairs (82 MB) 17.3 us; one token of 32 and 8 heads 3.6 us on the GPU.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/nvfp4.h"
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace rope {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxHeadDim = 512;
constexpr int kWarpsPerSm = 64;

struct Side {  // q or k
    const void *in;
    void *out;
    int64_t in_ld, out_ld;
    int32_t heads;
};

struct Call {
    Side side[2];
    const int64_t *positions;
    int64_t positions_ld;
    const nvfp4_rope_pair *pairs;
    int64_t tokens;
    int32_t axes, n_pairs, head_dim, adjacent;
    uint32_t parts;          // warps of a token
    int32_t heads_per_warp;
    float scale, sine;  // sine: scale, or its negative for the inverse
};

// A token's position on the axis of the lane's number, so that it is loaded beside the pairs and not behind them.
NVFP4_DEVINL int64_t lane_position(const Call &c, int64_t token, int lane)
{
    return lane < c.axes ? c.positions[lane * c.positions_ld + token] : 0;
}

// scale * (cos, +-sin) of a token's angle in one pair; the whole warp is here (`pair` beyond the last: anything).
NVFP4_DEVINL float2 turn_of(const Call &c, int64_t token, int64_t position, int pair)
{
    const bool there = pair < c.n_pairs;
    nvfp4_rope_pair p = {0, 0, 0};
    if (there)
        p = c.pairs[pair];
    const int axis = min((int)p.axis, c.axes - 1);
    int64_t at = __shfl_sync(0xFFFFFFFFu, position, axis & 31);
    if (axis >= 32)
        at = c.positions[axis * c.positions_ld + token];
    const uint64_t turn = (uint64_t)at * p.turn;
    // quarter turns and what is left of one: a multiple of 2^-32 turns, at most an eighth of one
    const uint32_t t = (uint32_t)((turn + (1ull << 31)) >> 32), quarter = (t + (1u << 29)) >> 30;
    float s, co;
    sincospif((float)(int32_t)(t - (quarter << 30)) * 0x1p-31f, &s, &co);
    if (quarter & 1) {
        const float x = co;
        co = -s;
        s = x;
    }
    if (quarter & 2) {
        co = -co;
        s = -s;
    }
    return make_float2(co * c.scale, s * c.sine);
}

NVFP4_DEVINL float load(const float *p) { return *p; }
NVFP4_DEVINL float load(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
NVFP4_DEVINL void store(float *p, float v) { *p = v; }
NVFP4_DEVINL void store(uint16_t *p, float v) { *p = f32_to_bf16(v); }

// Eight elements as they lie in memory: 16 bytes of bf16, 32 of fp32 (the loads of many heads are in flight together, and
// bf16 takes half the registers so).
template <class T> struct Eight;
template <> struct Eight<uint16_t> {
    uint4 w;

    NVFP4_DEVINL void load(const uint16_t *p) { w = *reinterpret_cast<const uint4 *>(p); }
    NVFP4_DEVINL void values(float (&x)[8]) const
    {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(v[j] << 16);
            x[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
        }
    }
};
template <> struct Eight<float> {
    float4 a, b;

    NVFP4_DEVINL void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    NVFP4_DEVINL void values(float (&x)[8]) const
    {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
NVFP4_DEVINL uint32_t pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
NVFP4_DEVINL void store8(uint16_t *p, const float (&x)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
}
NVFP4_DEVINL void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// A warp has one token and c.heads_per_warp heads of q and k (those of k behind those of q): lane = slot + slots * head
// turns the same 8 pairs of every (32 / slots)-th head, kBatch heads at most, with 16-byte loads and stores.  All its loads
// come before the cosines and sines, which pass through shared memory into registers.
template <class T> constexpr int kBatch = sizeof(T) == 2 ? 6 : 2;
constexpr int kTail = 2;

template <class T, bool ADJACENT>
__global__ void __launch_bounds__(kThreads) rope_kernel(Call c)
{
    __shared__ float2 turns[kWarps][kMaxHeadDim / 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // a programmatic dependent of the kernel before: nothing global is touched until that is done
    tc::griddep_launch_dependents();
    tc::griddep_wait();
    const uint32_t id = blockIdx.x * kWarps + warp;
    const uint32_t token = id / c.parts, part = id - token * c.parts;
    if (token >= c.tokens)
        return;
    const int slots = c.n_pairs / 8, step = 32 / slots, slot = lane % slots, first = lane / slots;
    const int begin = part * c.heads_per_warp, end = min(begin + c.heads_per_warp, c.side[0].heads + c.side[1].heads);
    const T *const q = static_cast<const T *>(c.side[0].in) + token * c.side[0].in_ld;
    const T *const k = static_cast<const T *>(c.side[1].in) + token * c.side[1].in_ld;
    T *const q_out = static_cast<T *>(c.side[0].out) + token * c.side[0].out_ld;
    T *const k_out = static_cast<T *>(c.side[1].out) + token * c.side[1].out_ld;
    const int a = ADJACENT ? 16 * slot : 8 * slot, b = ADJACENT ? a + 8 : a + c.n_pairs;
    constexpr int B = kBatch<T>;
    Eight<T> x[B], y[B];
    const int64_t position = lane_position(c, token, lane);
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const int h = begin + first + i * step, hk = h - c.side[0].heads;
        const T *in = hk < 0 ? q + h * c.head_dim : k + hk * c.head_dim;
        if (first < step && h < end) {
            x[i].load(in + a);
            y[i].load(in + b);
        }
    }
    // what is not turned, eight elements at a time and kTail of those in flight
    const int rest = c.head_dim / 8 - 2 * slots, n_rest = (end - begin) * rest;
    Eight<T> tail[kTail];
    const auto place = [&](int i, const T **in, T **out) {
        const int h = i / rest, at = (2 * slots + i - h * rest) * 8, hk = begin + h - c.side[0].heads;
        *in = (hk < 0 ? q + (begin + h) * c.head_dim : k + hk * c.head_dim) + at;
        *out = (hk < 0 ? q_out + (begin + h) * c.head_dim : k_out + hk * c.head_dim) + at;
        return *in != *out;
    };
    const auto load_tail = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kTail; ++j) {
            const T *in;
            T *out;
            if (i0 + 32 * j < n_rest && place(i0 + 32 * j, &in, &out))
                tail[j].load(in);
        }
    };
    load_tail(lane);
    for (int p = lane; p < (c.n_pairs + 31) / 32 * 32; p += 32) {
        const float2 t = turn_of(c, token, position, p);
        if (p < c.n_pairs)
            turns[warp][p] = t;
    }
    __syncwarp();
    float co[8], si[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 t = turns[warp][8 * slot + j];
        co[j] = t.x;
        si[j] = t.y;
    }
    if (first < step) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int h = begin + first + i * step, hk = h - c.side[0].heads;
            T *out = hk < 0 ? q_out + h * c.head_dim : k_out + hk * c.head_dim;
            if (h >= end)
                break;
            float m[8], n[8], u[8], v[8];
            x[i].values(m);
            y[i].values(n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (ADJACENT) {  // pair j: elements 2 j and 2 j + 1 of 16
                    const float xa = j < 4 ? m[(2 * j) & 7] : n[(2 * j) & 7], xb = j < 4 ? m[(2 * j + 1) & 7] : n[(2 * j + 1) & 7];
                    (j < 4 ? u : v)[(2 * j) & 7] = xa * co[j] - xb * si[j];
                    (j < 4 ? u : v)[(2 * j + 1) & 7] = xa * si[j] + xb * co[j];
                } else {
                    u[j] = m[j] * co[j] - n[j] * si[j];
                    v[j] = m[j] * si[j] + n[j] * co[j];
                }
            }
            store8(out + a, u);
            store8(out + b, v);
        }
    }
#pragma unroll 1
    for (int i0 = lane; i0 < n_rest; i0 += kTail * 32) {
        if (i0 != lane)
            load_tail(i0);
#pragma unroll
        for (int j = 0; j < kTail; ++j) {
            const T *in;
            T *out;
            float w[8];
            if (i0 + 32 * j < n_rest && place(i0 + 32 * j, &in, &out)) {
                tail[j].values(w);
                store8(out, w);
            }
        }
    }
}

// Any number of pairs: a warp has one token and c.heads_per_warp heads of q and k as above, whose pairs (and elements that are
// not turned) its lanes take one after the other, kAny pairs at a time.  8192 tokens of 40 and 8 bf16 heads of 80, 20 pairs:
// 62 us (8 at a time 68, with all heads to one warp and a pair at a time 66), 2000 of 16 and 16 fp32 heads 18.3 (54), one token
// 4.3 (36).  An element to a load, so it is bound by instructions.
constexpr int kAny = 4;

template <class T>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(Call c)
{
    __shared__ float2 turns[kWarps][kMaxHeadDim / 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    tc::griddep_launch_dependents();
    tc::griddep_wait();
    const int64_t id = (int64_t)blockIdx.x * kWarps + warp, token = id / c.parts;
    if (token >= c.tokens)
        return;
    const int begin = (int)(id - token * c.parts) * c.heads_per_warp, end = min(begin + c.heads_per_warp, c.side[0].heads + c.side[1].heads);
    const int64_t position = lane_position(c, token, lane);
    for (int p = lane; p < (c.n_pairs + 31) / 32 * 32; p += 32) {
        const float2 t = turn_of(c, token, position, p);
        if (p < c.n_pairs)
            turns[warp][p] = t;
    }
    __syncwarp();
    const int nq = c.side[0].heads, dim = c.head_dim;
    const T *const q = static_cast<const T *>(c.side[0].in) + token * c.side[0].in_ld;
    const T *const k = static_cast<const T *>(c.side[1].in) + token * c.side[1].in_ld;
    T *const q_out = static_cast<T *>(c.side[0].out) + token * c.side[0].out_ld;
    T *const k_out = static_cast<T *>(c.side[1].out) + token * c.side[1].out_ld;
    // f(number, whether of q, element of the token's q or k from which on, i) for each i of [0, width) of the heads, kAny of them
    // at a time: first `loads`, then `stores`
    const auto each = [&](int width, auto &&loads, auto &&stores) {
        int h = begin + lane / width, i = lane % width;
        while (__any_sync(0xFFFFFFFFu, h < end)) {
            int hs[kAny], is[kAny];
#pragma unroll
            for (int n = 0; n < kAny; ++n) {
                hs[n] = h;
                is[n] = i;
                if (h < end)
                    loads(n, h < nq, (h < nq ? h : h - nq) * dim, i);
                for (i += 32; i >= width; i -= width)
                    ++h;
            }
#pragma unroll
            for (int n = 0; n < kAny; ++n)
                if (hs[n] < end)
                    stores(n, hs[n] < nq, (hs[n] < nq ? hs[n] : hs[n] - nq) * dim, is[n]);
        }
    };
    const int step = c.adjacent ? 2 : 1, apart = c.adjacent ? 1 : c.n_pairs;  // from pair to pair, within one
    if (c.n_pairs > 0) {
        float x[kAny], y[kAny];
        each(
            c.n_pairs,
            [&](int n, bool of_q, int at, int p) {
                const T *in = (of_q ? q : k) + at + step * p;
                x[n] = load(in);
                y[n] = load(in + apart);
            },
            [&](int n, bool of_q, int at, int p) {
                const float2 t = turns[warp][p];
                T *out = (of_q ? q_out : k_out) + at + step * p;
                store(out, x[n] * t.x - y[n] * t.y);
                store(out + apart, x[n] * t.y + y[n] * t.x);
            });
    }
    // what is not turned
    const int turned = 2 * c.n_pairs;
    if (turned < dim && (q != q_out || k != k_out)) {
        T rest[kAny];
        each(
            dim - turned, [&](int n, bool of_q, int at, int i) { rest[n] = (of_q ? q : k)[at + turned + i]; },
            [&](int n, bool of_q, int at, int i) {
                if (of_q ? q != q_out : k != k_out)
                    (of_q ? q_out : k_out)[at + turned + i] = rest[n];
            });
    }
}

template <class T>
cudaError_t launch(Call c, int num_sms, cudaStream_t stream)
{
    if (c.n_pairs % 8 != 0 || c.n_pairs == 0 || c.n_pairs > 256) {
        // few tokens: a token's heads to as many warps as fill the GPU
        const int all = c.side[0].heads + c.side[1].heads;
        const int64_t fill = ((int64_t)num_sms * kWarpsPerSm + c.tokens - 1) / c.tokens;
        c.heads_per_warp = (int)((all + fill - 1) / fill);
        c.parts = (all + c.heads_per_warp - 1) / c.heads_per_warp;
        return launch_dependent(rope_any_kernel<T>, dim3((unsigned)((c.tokens * c.parts + kWarps - 1) / kWarps)), kThreads, 0, stream, c);
    }
    // A warp takes as many heads as its lanes load at once (kBatch rounds of heads, and never more); fewer, down to one each, while there are fewer than kWarpsPerSm
    // warps an SM (4999 tokens of 32 fp32 heads: 20.0 us at 24, 18.0 at 64, 17.9 at 128, where 8192 tokens of 48 bf16 heads
    // take 37.1 instead of 33.7).
    const int heads = c.side[0].heads + c.side[1].heads, round = 32 / (c.n_pairs / 8), most = (heads + round - 1) / round;
    const int least = (most + kBatch<T> - 1) / kBatch<T>;
    const int64_t want = ((int64_t)num_sms * kWarpsPerSm + c.tokens - 1) / c.tokens;
    c.parts = (int)(want < least ? least : want < most ? want : most);
    c.heads_per_warp = (most + c.parts - 1) / c.parts * round;
    c.parts = (heads + c.heads_per_warp - 1) / c.heads_per_warp;
    const dim3 grid((unsigned)((c.tokens * c.parts + kWarps - 1) / kWarps));
    return c.adjacent ? launch_dependent(rope_kernel<T, true>, grid, kThreads, 0, stream, c)
                      : launch_dependent(rope_kernel<T, false>, grid, kThreads, 0, stream, c);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool side_ok(const void *in, int64_t in_ld, const void *out, int64_t out_ld, int32_t heads, const nvfp4_rope_args *a)
{
    const int64_t width = (int64_t)heads * a->head_dim;
    const int unit = a->dtype == NVFP4_OUT_BF16 ? 8 : 4;
    if (in == out && in_ld != out_ld && a->n_tokens > 1)  // in place, but a row would overwrite others
        return false;
    return in && out && aligned(in, 16) && aligned(out, 16) && in_ld >= width && out_ld >= width && in_ld % unit == 0 &&
           out_ld % unit == 0 && in_ld <= (INT64_C(1) << 60) / a->n_tokens && out_ld <= (INT64_C(1) << 60) / a->n_tokens;
}

}  // namespace rope
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_rope_pairs(const double *inv_freq, const int32_t *axis, int32_t n_pairs, nvfp4_rope_pair *pairs)
{
    if (n_pairs < 0 || (n_pairs > 0 && (!inv_freq || !pairs)))
        return NVFP4_ERR_INVALID_ARG;
    // 2^192 / (2 pi), from its low 64 bits on
    static const uint64_t kTurn[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};
    for (int i = 0; i < n_pairs; ++i) {
        if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) >= 0x1p31 || (axis && (axis[i] < 0 || axis[i] > 255)))
            return NVFP4_ERR_INVALID_ARG;
        // |inv_freq| = m * 2^e with a 53-bit m; its turn is m * 2^192 / (2 pi) / 2^(128 - e), rounded to nearest
        int e;
        const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(inv_freq[i]), &e), 53);
        const int shift = 128 - (e - 53);
        uint64_t limb[4], carry = 0;
        for (int j = 0; j < 3; ++j) {
            const unsigned __int128 t = (unsigned __int128)m * kTurn[j] + carry;
            limb[j] = (uint64_t)t;
            carry = (uint64_t)(t >> 64);
        }
        limb[3] = carry;
        const auto bits_from = [&](int at) -> uint64_t {  // 64 bits of the product from bit `at` on
            if (at >= 256)
                return 0;
            const int w = at / 64, r = at % 64;
            uint64_t v = limb[w] >> r;
            if (r && w < 3)
                v |= limb[w + 1] << (64 - r);
            return v;
        };
        uint64_t turn = bits_from(shift) + (bits_from(shift - 1) & 1);
        if (std::signbit(inv_freq[i]))
            turn = 0 - turn;
        pairs[i].turn = turn;
        pairs[i].axis = axis ? (uint32_t)axis[i] : 0;
        pairs[i].reserved = 0;
    }
    return NVFP4_OK;
}

int nvfp4_rope(const nvfp4_rope_args *args, nvfp4_stream_t stream)
{
    const nvfp4_rope_args *a = args;
    if (!a || a->n_tokens < 0 || (a->dtype != NVFP4_OUT_F32 && a->dtype != NVFP4_OUT_BF16) ||
        (a->adjacent != 0 && a->adjacent != 1) || (a->inverse != 0 && a->inverse != 1) || !std::isfinite(a->scale))
        return NVFP4_ERR_INVALID_ARG;
    if (a->head_dim < 8 || a->head_dim > rope::kMaxHeadDim || a->head_dim % 8 != 0 || a->n_pairs < 0 ||
        2 * a->n_pairs > a->head_dim || a->n_axes < 1 || a->n_axes > 256 || a->n_q_heads < 0 || a->n_k_heads < 0 ||
        a->n_q_heads > 8192 || a->n_k_heads > 8192 || a->n_tokens >= INT64_C(1) << 31)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (a->n_tokens == 0 || a->n_q_heads + a->n_k_heads == 0)
        return NVFP4_OK;
    if (!a->positions || !rope::aligned(a->positions, 8) ||
        (a->n_axes > 1 && ((a->positions_ld < a->n_tokens && a->positions_ld != 0) || a->positions_ld > (INT64_C(1) << 60) / a->n_axes)) ||
        (a->n_pairs > 0 && (!a->pairs || !rope::aligned(a->pairs, 16))))
        return NVFP4_ERR_INVALID_ARG;
    if ((a->n_q_heads > 0 && !rope::side_ok(a->q, a->q_ld, a->q_out, a->q_out_ld, a->n_q_heads, a)) ||
        (a->n_k_heads > 0 && !rope::side_ok(a->k, a->k_ld, a->k_out, a->k_out_ld, a->n_k_heads, a)))
        return NVFP4_ERR_INVALID_ARG;
    rope::Call c;
    c.side[0] = {a->q, a->q_out, a->q_ld, a->q_out_ld, a->n_q_heads};
    c.side[1] = {a->k, a->k_out, a->k_ld, a->k_out_ld, a->n_k_heads};
    c.positions = a->positions;
    c.positions_ld = a->n_axes > 1 ? a->positions_ld : 0;
    c.pairs = a->pairs;
    c.tokens = a->n_tokens;
    c.axes = a->n_axes;
    c.n_pairs = a->n_pairs;
    c.head_dim = a->head_dim;
    c.adjacent = a->adjacent;
    c.scale = a->scale;
    c.sine = a->inverse ? -a->scale : a->scale;
    int sms = 0;
    const int rc = current_num_sms(&sms);
    if (rc != NVFP4_OK)
        return rc;
    const cudaError_t e = a->dtype == NVFP4_OUT_BF16 ? rope::launch<uint16_t>(c, sms, (cudaStream_t)stream)
                                                     : rope::launch<float>(c, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // extern "C"
