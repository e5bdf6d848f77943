// attention.cu -- attention of new tokens over the quantised paged KV cache
// (nvfp4_paged_attention; include/nvfp4.h has the definition).
#include <cmath>
#include <cstdint>

#include "attention.h"
#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace attn {

namespace {

constexpr int kWarps = 4;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// D / 32 consecutive elements (from element `at`) of row `row` of a block, as
// codes times block scales in fp32; the row's exponent is not applied.
template <int FMT, int D>
NVFP4_DEVINL void load_elems(const uint8_t *blk, int page_shift, int row, int at, float (&x)[D / 32])
{
    using R = kv::Row<FMT, D>;
    if constexpr (FMT == NVFP4_KV_E4M3) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            x[i] = e4m3_to_f32(blk[row * R::kCode + at + i]);
    } else {
        const float s = e4m3_to_f32(blk[(R::kCode << page_shift) + row * R::kScale + at / 16]);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t code = blk[row * R::kCode + (at + i) / 2] >> ((at + i) % 2 * 4) & 15u;
            const float mag[8] = {0.f, .5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
            x[i] = (code & 8 ? -1.f : 1.f) * mag[code & 7] * s;
        }
    }
}

// One warp per (new token, query head), one key at a time: the plain form of
// the operator, in fp32 throughout.
template <int FMT, int D>
__global__ void __launch_bounds__(32 * kWarps) attention_rows_kernel(Call c)
{
    using R = kv::Row<FMT, D>;
    constexpr int E = D / 32;
    const int lane = threadIdx.x % 32;
    const int64_t id = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const int row = (int)(id / c.q_heads), head = (int)(id % c.q_heads);
    if (row >= c.total_q)
        return;
    int b = 0;
    if (c.q_offsets) {
        int last = c.n_seqs;  // the sequence whose range holds `row`
        while (last - b > 1) {
            const int mid = (b + last) / 2;
            if (c.q_offsets[mid] <= row)
                b = mid;
            else
                last = mid;
        }
    } else {
        b = row / c.max_q_len;
    }
    const Seq s = load_seq(c, b);
    const int i = row - s.q_begin;
    if (i < 0 || i >= s.n)
        return;
    int lo, hi;
    key_range(c, s, i, &lo, &hi);
    const uint64_t bits = c.tree ? c.tree[row] : 0;
    float q[E];
#pragma unroll
    for (int d = 0; d < E; ++d) {
        const float x = __uint_as_float((uint32_t)c.q[(int64_t)row * c.q_ld + head * D + lane * E + d] << 16);
        q[d] = isfinite(x) ? x : NAN;  // an infinity times K would depend on K's signs
    }
    float top = -INFINITY, sum = 0.f, o[E] = {};
    for (int j = lo; j < hi; ++j) {
        if (c.tree && j >= s.past && (j - s.past >= 64 || !(bits >> (j - s.past) & 1)))
            continue;
        const int page = page_of(c, b, j);
        if (page < 0)
            continue;
        const int at = j & ((1 << c.pool.page_shift) - 1);
        const uint8_t *kb = kv::block_ptr(c.pool, page, head / c.group, 0);
        const uint8_t *vb = kv::block_ptr(c.pool, page, head / c.group, 1);
        float x[E], dot = 0.f;
        load_elems<FMT, D>(kb, c.pool.page_shift, at, lane * E, x);
#pragma unroll
        for (int d = 0; d < E; ++d)
            dot += q[d] * x[d];
#pragma unroll
        for (int off = 16; off > 0; off /= 2)
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
        const int exps = (R::kCode + R::kScale) << c.pool.page_shift;
        const float t = dot * kv::exp2_byte(kb[exps + at]) * c.scale_log2;
        const float next = fmaxf(top, t);
        const float shrink = top == -INFINITY ? 0.f : exp2f(top - next);
        const float p = next == -INFINITY ? (t == t ? 0.f : t) : exp2f(t - next);
        load_elems<FMT, D>(vb, c.pool.page_shift, at, lane * E, x);
        const float pv = p * kv::exp2_byte(vb[exps + at]);
        sum = sum * shrink + p;
#pragma unroll
        for (int d = 0; d < E; ++d)
            o[d] = o[d] * shrink + pv * x[d];
        top = next;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int d = 0; d < E; ++d) {
        const int64_t at = (int64_t)row * c.out_ld + head * D + lane * E + d;
        if (c.out_bf16)
            static_cast<uint16_t *>(c.out)[at] = f32_to_bf16(o[d] * inv);
        else
            static_cast<float *>(c.out)[at] = o[d] * inv;
    }
}

template <class F>
void by_format(int format, int head_dim, F &&f)
{
    using std::integral_constant;
    if (format == NVFP4_KV_E4M3)
        head_dim == 64 ? f(integral_constant<int, 0>{}, integral_constant<int, 64>{})
                       : f(integral_constant<int, 0>{}, integral_constant<int, 128>{});
    else
        head_dim == 64 ? f(integral_constant<int, 1>{}, integral_constant<int, 64>{})
                       : f(integral_constant<int, 1>{}, integral_constant<int, 128>{});
}

// Sizes alone; what nvfp4_paged_attention_workspace_bytes looks at.
int check_sizes(const nvfp4_paged_attention_args *a)
{
    if (a->n_seqs < 0 || a->total_q < 0 || a->max_q_len < 0)
        return NVFP4_ERR_INVALID_ARG;
    if (nvfp4_kv_page_bytes(a->cache.page_size, a->cache.n_kv_heads, a->cache.head_dim, a->cache.format) == 0)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (a->n_seqs > 65535 || a->total_q > INT32_MAX / 8192 || a->max_q_len > a->total_q)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (a->n_q_heads < 1 || a->n_q_heads > 8192 || a->n_q_heads % a->cache.n_kv_heads != 0)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    return NVFP4_OK;
}

int check_args(const nvfp4_paged_attention_args *a)
{
    if (!a)
        return NVFP4_ERR_INVALID_ARG;
    const int rc = check_sizes(a);
    if (rc != NVFP4_OK)
        return rc;
    if (a->out_dtype != NVFP4_OUT_F32 && a->out_dtype != NVFP4_OUT_BF16)
        return NVFP4_ERR_INVALID_ARG;
    if ((a->causal != 0 && a->causal != 1) || a->window < 0 || !std::isfinite(a->scale))
        return NVFP4_ERR_INVALID_ARG;
    if (a->window > 0 && !a->causal)
        return NVFP4_ERR_INVALID_ARG;
    if (a->tree && (!a->causal || a->window > 0))
        return NVFP4_ERR_INVALID_ARG;
    if (a->tree && a->max_q_len > 64)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!a->q_offsets && a->n_seqs * a->max_q_len != a->total_q)
        return NVFP4_ERR_INVALID_ARG;
    if (a->total_q == 0 || a->n_seqs == 0)
        return NVFP4_OK;
    const int64_t width = (int64_t)a->n_q_heads * a->cache.head_dim;
    if (a->q_ld < width || a->out_ld < width || a->q_ld % 8 != 0 || a->out_ld % 8 != 0 ||
        a->q_ld > (INT64_C(1) << 60) / a->total_q || a->out_ld > (INT64_C(1) << 60) / a->total_q)
        return NVFP4_ERR_INVALID_ARG;
    if (a->table_width < 0 || a->table_width > (INT64_C(1) << 31) / a->cache.page_size)
        return NVFP4_ERR_INVALID_ARG;
    if (!a->q || !a->out || !a->kv_lens || (a->table_width > 0 && !a->block_table))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->kv_lens, 4) || !aligned(a->block_table, 4) ||
        !aligned(a->q_offsets, 4) || !aligned(a->tree, 8))
        return NVFP4_ERR_INVALID_ARG;
    return NVFP4_OK;
}

}  // namespace
}  // namespace attn
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_paged_attention_workspace_bytes(const nvfp4_paged_attention_args *args)
{
    if (!args || attn::check_sizes(args) != NVFP4_OK)
        return 0;
    return kKvWorkspaceBytes;
}

int nvfp4_paged_attention(const nvfp4_paged_attention_args *args, void *workspace, size_t workspace_bytes,
                          nvfp4_stream_t stream)
{
    int rc = attn::check_args(args);
    if (rc != NVFP4_OK)
        return rc;
    attn::Call c;
    if (workspace_bytes < nvfp4_paged_attention_workspace_bytes(args))
        return NVFP4_ERR_WORKSPACE;
    if (!workspace)
        return NVFP4_ERR_INVALID_ARG;
    rc = kv::make_pool(&args->cache, workspace, workspace_bytes, &c.pool);
    if (rc != NVFP4_OK || args->total_q == 0 || args->n_seqs == 0)
        return rc;
    c.q = args->q;
    c.q_ld = args->q_ld;
    c.out = args->out;
    c.out_ld = args->out_ld;
    c.table = args->block_table;
    c.table_width = args->table_width;
    c.kv_lens = args->kv_lens;
    c.q_offsets = args->q_offsets;
    c.tree = args->tree;
    c.n_seqs = (int32_t)args->n_seqs;
    c.total_q = (int32_t)args->total_q;
    c.max_q_len = (int32_t)args->max_q_len;
    c.q_heads = args->n_q_heads;
    c.group = args->n_q_heads / args->cache.n_kv_heads;
    c.window = args->window > INT32_MAX ? 0 : (int32_t)args->window;
    c.out_bf16 = args->out_dtype == NVFP4_OUT_BF16;
    c.causal = args->causal;
    c.scale_log2 = args->scale * 1.4426950408889634f;
    const int64_t warps = args->total_q * args->n_q_heads;
    const uint32_t grid = (uint32_t)((warps + attn::kWarps - 1) / attn::kWarps);
    attn::by_format(args->cache.format, args->cache.head_dim, [&](auto fmt, auto d) {
        attn::attention_rows_kernel<fmt.value, d.value><<<grid, 32 * attn::kWarps, 0, (cudaStream_t)stream>>>(c);
    });
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // extern "C"
