// prompt_attention.h -- what the kernels of nvfp4_prompt_attention get.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {
namespace prompt {

constexpr int kMaxGroup = 128;  // query heads of a KV head

struct Call {
    const uint16_t *q, *k, *v;
    void *out;
    int64_t q_ld, k_ld, v_ld, out_ld;
    const int32_t *offsets;  // or null: one sequence
    uint32_t *status;        // device status word, or null
    int32_t n_seqs, total, window;
    int32_t q_heads, kv_heads, group;
    int32_t causal, out_bf16;
    float scale_log2;        // scores in powers of two
};

}  // namespace prompt
}  // namespace nvfp4
