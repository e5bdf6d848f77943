// attention.cu -- attention of new tokens over the quantised paged KV cache
// (nvfp4_paged_attention; include/nvfp4.h has the definition).
#include <cmath>
#include <cstdint>

#include "attention_plan.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace attn {

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Which kernel: by the rows that share a KV head's keys.  At 32 rows the chunk
// kernel takes 38.0 us where the decode kernel took 42.3 in 32-row items (8 sequences
// of 4000 E4M3 keys, 32 and 8 heads) and 62.9 where it took 69.2 (32 of 2000 NVFP4), but
// 74.4 where it took 73.1 (32 of 2000 E4M3) and 45.8 where it took 38.3 (one of 30000);
// at 24 rows 38.0 against 34.4 and 46.1 against 31.1.  fp32 outputs keep the decode
// kernel's wide weights.
bool use_chunk(int64_t rows, int out_dtype) { return rows > 24 && out_dtype == NVFP4_OUT_BF16; }

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
    if (a->table_width < 0 || a->table_width > INT64_C(0x7FFFF000) / a->cache.page_size)
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
    const int64_t rows = args->max_q_len * (args->n_q_heads / args->cache.n_kv_heads);
    const bool chunk = attn::use_chunk(rows, NVFP4_OUT_BF16);  // the larger of the two types' needs
    const int block = !chunk ? attn::decode_block(rows) : rows <= 128 ? 128 : 256;
    const int ctas = chunk ? attn::kMaxChunkCtas : attn::decode_max_ctas(block);
    return attn::kPartialOffset + (size_t)ctas * 2 * block * (args->cache.head_dim + 2) * sizeof(float);
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
    c.item_cost = 0;
    c.out_bf16 = args->out_dtype == NVFP4_OUT_BF16;
    c.causal = args->causal;
    c.scale_log2 = args->scale * 1.4426950408889634f;
    int sms = 0;
    rc = current_num_sms(&sms);
    if (rc != NVFP4_OK)
        return rc;
    const bool e4m3 = args->cache.format == NVFP4_KV_E4M3;
    const auto launch = attn::use_chunk((int64_t)c.max_q_len * c.group, args->out_dtype)
                            ? (e4m3 ? attn::launch_chunk_e4m3 : attn::launch_chunk_nvfp4)
                            : (e4m3 ? attn::launch_decode_e4m3 : attn::launch_decode_nvfp4);
    const cudaError_t e = launch(c, args->cache.head_dim, workspace, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // extern "C"
