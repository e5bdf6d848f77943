// prompt_attention.cu -- attention of packed whole prompts over their own K and V
// (nvfp4_prompt_attention; include/nvfp4.h has the definition).
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "kv_layout.cuh"
#include "prompt_attention.h"

namespace nvfp4 {
namespace prompt {

namespace {

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

// One warp per token and query head: its keys one by one.
template <int D>
__global__ void __launch_bounds__(128) row_kernel(Call c)
{
    const int lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    const int token = (int)(row / c.q_heads), head = (int)(row % c.q_heads);
    if (token >= c.total)
        return;
    int begin = 0, end = c.offsets ? 0 : c.total;
    for (int b = 0; c.offsets && b < c.n_seqs; ++b) {
        const int from = c.offsets[b], to = c.offsets[b + 1];
        if (from < 0 || to < from || to > c.total) {
            if (row == 0 && lane == 0)
                kv::report_index(c.status, kStatusPromptOffsets);
        } else if (token >= from && token < to) {
            begin = from;
            end = to;
        }
    }
    if (token >= end)
        return;
    const int lo = c.window > 0 ? max(begin, token + 1 - c.window) : begin, hi = c.causal ? token + 1 : end;
    constexpr int E = D / 32;
    const auto element = [](const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); };
    const int64_t kv = (int64_t)(head / c.group) * D + lane;
    float q[E], acc[E], top = -INFINITY, sum = 0.f;
    for (int e = 0; e < E; ++e) {
        q[e] = element(c.q + token * c.q_ld + (int64_t)head * D + lane + 32 * e) * c.scale_log2;
        acc[e] = 0.f;
    }
    for (int j = lo; j < hi; ++j) {
        float s = 0.f;
        for (int e = 0; e < E; ++e)
            s = fmaf(q[e], element(c.k + j * c.k_ld + kv + 32 * e), s);
        for (int o = 16; o > 0; o /= 2)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        const float next = fmaxf(top, s), base = next == -INFINITY ? 0.f : next;
        const float shrink = exp2f(top - base), w = exp2f(s - base);
        top = next;
        sum = fmaf(sum, shrink, w);
        for (int e = 0; e < E; ++e)
            acc[e] = fmaf(acc[e], shrink, w * element(c.v + j * c.v_ld + kv + 32 * e));
    }
    for (int e = 0; e < E; ++e) {
        const int64_t at = token * c.out_ld + (int64_t)head * D + lane + 32 * e;
        if (c.out_bf16)
            static_cast<uint16_t *>(c.out)[at] = f32_to_bf16(acc[e] / sum);
        else
            static_cast<float *>(c.out)[at] = acc[e] / sum;
    }
}

}  // namespace
}  // namespace prompt
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int nvfp4_prompt_attention(const nvfp4_prompt_attention_args *args, void *workspace, size_t workspace_bytes,
                                      nvfp4_stream_t stream)
{
    const int rc = prompt::check_args(args);
    if (rc != NVFP4_OK)
        return rc;
    if (workspace && !prompt::aligned(workspace, 16))
        return NVFP4_ERR_INVALID_ARG;
    if (workspace && workspace_bytes < kKvWorkspaceBytes)
        return NVFP4_ERR_WORKSPACE;
    if (args->total == 0 || args->n_seqs == 0)
        return NVFP4_OK;
    prompt::Call c;
    c.q = args->q;
    c.k = args->k;
    c.v = args->v;
    c.out = args->out;
    c.q_ld = args->q_ld;
    c.k_ld = args->k_ld;
    c.v_ld = args->v_ld;
    c.out_ld = args->out_ld;
    c.offsets = args->offsets;
    c.status = workspace ? reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + kStatusWordOffset) : nullptr;
    c.n_seqs = (int32_t)args->n_seqs;
    c.total = (int32_t)args->total;
    c.window = args->window > INT32_MAX ? 0 : (int32_t)args->window;
    c.q_heads = args->n_q_heads;
    c.kv_heads = args->n_kv_heads;
    c.group = args->n_q_heads / args->n_kv_heads;
    c.causal = args->causal;
    c.out_bf16 = args->out_dtype == NVFP4_OUT_BF16;
    c.scale_log2 = args->scale * 1.4426950408889634f;
    const unsigned blocks = (unsigned)(((int64_t)c.total * c.q_heads + 3) / 4);
    if (args->head_dim == 64)
        prompt::row_kernel<64><<<blocks, 128, 0, (cudaStream_t)stream>>>(c);
    else
        prompt::row_kernel<128><<<blocks, 128, 0, (cudaStream_t)stream>>>(c);
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
