// kv_layout.cuh -- the quantised paged KV cache as kernels see it: where a
// row's codes, scales and exponent lie (include/nvfp4.h has the format).
#pragma once

#include "../../include/nvfp4.h"
#include "common.cuh"

namespace nvfp4 {
namespace kv {

// A cache's pool and the sizes that every address is made of.
struct Pool {
    uint8_t *base;
    int64_t n_pages;
    int64_t page_bytes;    // every head, K and V
    int32_t block_bytes;   // one head's K (or V) rows of one page
    int32_t page_shift;    // page_size = 1 << page_shift
    int32_t heads;
    uint32_t *status;      // device status word, or null
};

template <int FMT, int D>
struct Row {
    static constexpr int kCode = FMT == NVFP4_KV_E4M3 ? D : D / 2;    // bytes of codes
    static constexpr int kScale = FMT == NVFP4_KV_E4M3 ? 0 : D / 16;  // bytes of block scales
    static constexpr int kBytes = kCode + kScale + 1;
    static constexpr float kTop = FMT == NVFP4_KV_E4M3 ? 448.f : 2688.f;  // largest value at e = 127
};

constexpr int kExpMin = -100, kExpMax = 100;  // range of the row exponent
constexpr uint32_t kNanRow = 255;

// Block of (page, head, K or V); `page` is within the pool.
NVFP4_DEVINL uint8_t *block_ptr(const Pool &p, int64_t page, int head, int is_v)
{
    return p.base + page * p.page_bytes + (int64_t)(head * 2 + is_v) * p.block_bytes;
}

// Stores the code of an index outside its bounds, unless the status word holds one
// already: a timeout's must stay, since it tells that the workspace is not clean.
NVFP4_DEVINL void report_index(uint32_t *status, uint32_t code)
{
    if (status)
        atomicCAS(status, 0u, code);
}
// Stores the code of a wait that ran out.
NVFP4_DEVINL void report_timeout(uint32_t *status, uint32_t code)
{
    if (status)
        atomicExch(status, code);
}

// 2^(e - 127) as a float; NaN for the mark of a row that is not a number.
NVFP4_DEVINL float exp2_byte(uint32_t e) { return __uint_as_float(e == kNanRow ? 0x7FC00000u : e << 23); }

// Four E4M3 bytes with those that are not a number (0x7F, 0xFF; the append
// writes none) replaced by zeros.
NVFP4_DEVINL uint32_t without_nan(uint32_t w)
{
    const uint32_t t = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return w & ~((t >> 7) * 0xFFu);
}

// Host: checks of a cache's description, and its Pool.  0, or an nvfp4_status.
int make_pool(const nvfp4_kv_cache *c, void *workspace, size_t workspace_bytes, Pool *out);

}  // namespace kv
}  // namespace nvfp4
