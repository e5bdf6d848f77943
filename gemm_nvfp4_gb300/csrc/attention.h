// attention.h -- launch interface between the checks of nvfp4_paged_attention
// (attention.cu) and its kernels.  Internal to libnvfp4.so.
#pragma once

#include "kernels.h"
#include "kv_layout.cuh"

namespace nvfp4 {
namespace attn {

// A checked call as the kernels see it.
struct Call {
    kv::Pool pool;
    const uint16_t *q;
    int64_t q_ld;
    void *out;
    int64_t out_ld;
    const int32_t *table;
    int64_t table_width;
    const int32_t *kv_lens;
    const int32_t *q_offsets;
    const uint64_t *tree;
    int32_t n_seqs, total_q, max_q_len;
    int32_t q_heads, group;  // query heads, query heads of one KV head
    int32_t window;          // 0: none
    int32_t item_cost;       // attention_plan.cuh
    int32_t out_bf16, causal;
    float scale_log2;  // scale * log2(e): the softmax works in powers of two
};

// One sequence of a call, clamped to what the call's buffers hold.
struct Seq {
    int32_t q_begin;  // first row of q
    int32_t n;        // new tokens
    int32_t kv;       // keys
    int32_t past;     // causal: position of the first new token
};

NVFP4_DEVINL Seq load_seq(const Call &c, int b)
{
    Seq s;
    bool bad = false;
    if (c.q_offsets) {
        const int lo = c.q_offsets[b], hi = c.q_offsets[b + 1];
        bad |= lo < 0 || hi < lo || hi > c.total_q;
        s.q_begin = min(max(lo, 0), c.total_q);
        s.n = min(max(hi, s.q_begin), c.total_q) - s.q_begin;
    } else {
        s.q_begin = b * c.max_q_len;
        s.n = c.max_q_len;
    }
    bad |= s.n > c.max_q_len;
    s.n = min(s.n, c.max_q_len);
    const int kv = c.kv_lens[b];
    const int64_t room = c.table_width << c.pool.page_shift;
    bad |= kv < 0 || kv > room;
    s.kv = (int)min((int64_t)max(kv, 0), room);
    s.past = s.kv - s.n;
    if (c.causal && s.past < 0) {
        // fewer keys than new tokens: the first tokens see nothing
        bad = true;
    }
    if (bad)
        kv::report_index(c.pool.status, kStatusKvAttention);
    return s;
}

// Keys [lo, hi) that new token i of a sequence may see (tree: before its mask).
NVFP4_DEVINL void key_range(const Call &c, const Seq &s, int i, int *lo, int *hi)
{
    *lo = 0;
    *hi = s.kv;
    if (c.causal && !c.tree) {
        *hi = min(s.kv, max(0, s.past + i + 1));
        if (c.window > 0)
            *lo = max(0, s.past + i + 1 - c.window);
    }
}

// Few rows per KV head (attention_decode.cuh), by cache format.
cudaError_t launch_decode_e4m3(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream);
cudaError_t launch_decode_nvfp4(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream);
// Many rows per KV head, bf16 outputs (attention_chunk.cuh).
cudaError_t launch_chunk_e4m3(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream);
cudaError_t launch_chunk_nvfp4(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream);

}  // namespace attn
}  // namespace nvfp4
