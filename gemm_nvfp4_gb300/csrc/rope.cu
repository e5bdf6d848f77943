// rope.cu -- rotary positions with one position per axis and token (nvfp4_rope;
// include/nvfp4.h has the definition).
//
// An angle is position * frequency, and only its fraction of a turn counts.  In fp32
// that product is off by 0.06 radians at position 2^20; here a frequency is a 64-bit
// fixed-point fraction of a turn, made once on the host, and the product of the two
// integers modulo 2^64 is the angle's fraction with an error of |position| * 2^-65
// turns, for the price of one integer multiplication.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/nvfp4.h"
#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace rope {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxHeadDim = 512;

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
    float scale, sine;  // sine: scale, or its negative for the inverse
};

// scale * (cos, +-sin) of a token's angle in one pair.
NVFP4_DEVINL float2 turn_of(const Call &c, int64_t token, int pair)
{
    const nvfp4_rope_pair p = c.pairs[pair];
    const int axis = min((int)p.axis, c.axes - 1);
    const uint64_t turn = (uint64_t)c.positions[axis * c.positions_ld + token] * p.turn;
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

// One warp per token: the pairs' cosines and sines once, then every head.
template <class T>
__global__ void __launch_bounds__(kThreads) rope_kernel(Call c)
{
    __shared__ float2 turns[kWarps][kMaxHeadDim / 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t token = (int64_t)blockIdx.x * kWarps + warp;
    if (token >= c.tokens)
        return;
    for (int p = lane; p < c.n_pairs; p += 32)
        turns[warp][p] = turn_of(c, token, p);
    __syncwarp();
    for (int s = 0; s < 2; ++s) {
        const Side &side = c.side[s];
        for (int h = 0; h < side.heads; ++h) {
            const T *in = static_cast<const T *>(side.in) + token * side.in_ld + (int64_t)h * c.head_dim;
            T *out = static_cast<T *>(side.out) + token * side.out_ld + (int64_t)h * c.head_dim;
            for (int p = lane; p < c.n_pairs; p += 32) {
                const float2 t = turns[warp][p];
                const int a = c.adjacent ? 2 * p : p, b = c.adjacent ? 2 * p + 1 : p + c.n_pairs;
                const float x = load(in + a), y = load(in + b);
                store(out + a, x * t.x - y * t.y);
                store(out + b, x * t.y + y * t.x);
            }
            if (in != out)
                for (int i = 2 * c.n_pairs + lane; i < c.head_dim; i += 32)
                    out[i] = in[i];
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool side_ok(const void *in, int64_t in_ld, const void *out, int64_t out_ld, int32_t heads, const nvfp4_rope_args *a)
{
    const int64_t width = (int64_t)heads * a->head_dim;
    const int unit = a->dtype == NVFP4_OUT_BF16 ? 8 : 4;
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
        (a->n_axes > 1 && (a->positions_ld < a->n_tokens || a->positions_ld > (INT64_C(1) << 60) / a->n_axes)) ||
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
    const unsigned blocks = (unsigned)((a->n_tokens + rope::kWarps - 1) / rope::kWarps);
    if (a->dtype == NVFP4_OUT_BF16)
        rope::rope_kernel<uint16_t><<<blocks, rope::kThreads, 0, (cudaStream_t)stream>>>(c);
    else
        rope::rope_kernel<float><<<blocks, rope::kThreads, 0, (cudaStream_t)stream>>>(c);
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // extern "C"
