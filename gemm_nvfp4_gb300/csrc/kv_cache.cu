// kv_cache.cu -- rows into and out of the quantised paged KV cache
// (nvfp4_kv_append, nvfp4_kv_read; the format is in include/nvfp4.h).
//
// Both are copies with a change of format, bound by HBM for many tokens (a
// 128-element bf16 row of 256 B becomes 129 or 73 B) and by the launch for
// few.  D / 8 neighbouring lanes hold one row, 8 elements (one 16-byte vector
// of bf16) each: loads and stores of values are whole 16-byte vectors, a row's
// maximum takes 3 or 4 shuffles, and an NVFP4 block of 16 is two lanes.
#include <cstdint>

#include "kernels.h"
#include "kv_layout.cuh"

namespace nvfp4 {
namespace kv {

namespace {

constexpr int kThreads = 256;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Two fp32 -> two E4M3 bytes (lo in the low byte), nearest even.
NVFP4_DEVINL uint32_t f32x2_to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two E2M1 codes of a byte to f16x2, exact (low nibble in the low half).
NVFP4_DEVINL uint32_t e2m1x2_to_f16x2(uint32_t byte)
{
    uint32_t r;
    asm("{ .reg .b8 b, z; mov.b16 {b, z}, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(r) : "h"((uint16_t)byte));
    return r;
}

NVFP4_DEVINL float2 f16x2_to_f32(uint32_t h2)
{
    float2 f;
    asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h2));
    return f;
}

NVFP4_DEVINL uint32_t f32x2_to_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Smallest k with amax <= T * 2^k, at least kExpMin; amax is a finite bf16
// value given as fp32.  T = (1 + F / 2^23) * 2^E: amax has exponent x and
// fraction f, so k = x - E, one more if f > F.  (A bf16 subnormal or zero
// reads exponent field 0, hence k = kExpMin, which is where it belongs.)
template <int FMT>
NVFP4_DEVINL int row_exponent(float amax)
{
    constexpr uint32_t top = FMT == NVFP4_KV_E4M3 ? 0x43E00000u /* 448 */ : 0x45280000u /* 2688 */;
    const uint32_t b = __float_as_uint(amax);
    const int k = (int)(b >> 23) - (int)(top >> 23) + ((b & 0x7FFFFFu) > (top & 0x7FFFFFu) ? 1 : 0);
    return k < kExpMin ? kExpMin : k;
}

NVFP4_DEVINL float pow2f(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// Shared by both kernels: which row a group of lanes works on.  Rows are
// ordered (token, K or V, head), so a token's K rows are neighbours, as in k.
struct RowId {
    uint32_t token;
    int is_v, head;
};

NVFP4_DEVINL RowId row_id(uint32_t r, uint32_t heads)
{
    RowId id;
    id.token = r / (2 * heads);
    const uint32_t rest = r - id.token * 2 * heads;
    id.is_v = rest >= heads;
    id.head = (int)(rest - (id.is_v ? heads : 0));
    return id;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(Pool pool, const uint16_t *__restrict__ k, int64_t k_ld,
                                                          const uint16_t *__restrict__ v, int64_t v_ld,
                                                          const int64_t *__restrict__ slots, uint32_t n_rows)
{
    constexpr int L = D / 8;  // lanes of a row
    using R = Row<FMT, D>;
    const int lane = threadIdx.x % L;
    const uint32_t per_grid = gridDim.x * (kThreads / L);
    const uint32_t rounds = (n_rows + per_grid - 1) / per_grid;
    uint32_t r = blockIdx.x * (kThreads / L) + threadIdx.x / L;
    for (uint32_t it = 0; it < rounds; ++it, r += per_grid) {
        // every lane stays for the shuffles; rows beyond the end store nothing
        const bool live = r < n_rows;
        const RowId id = row_id(live ? r : 0, pool.heads);
        const int64_t slot = live ? slots[id.token] : -1;
        const uint16_t *src = id.is_v ? v + (int64_t)id.token * v_ld : k + (int64_t)id.token * k_ld;
        const uint4 x = ldg_v4(src + (int64_t)id.head * D + lane * 8);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        // maximum of the magnitudes as integers: NaN and infinity come out on top
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
        uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const uint32_t block_max = m;  // of this lane pair's 16 elements
#pragma unroll
        for (int o = 2; o < L; o *= 2)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (!live || slot < 0)
            continue;
        const int64_t page = slot >> pool.page_shift;
        if (page >= pool.n_pages) {
            if (lane == 0)
                report(pool.status, kStatusKvAppendSlot);
            continue;
        }
        const int at = (int)(slot & ((1 << pool.page_shift) - 1));
        int ke = row_exponent<FMT>(__uint_as_float(m << 16));
        const bool bad = m >= 0x7F80u || ke > kExpMax;
        const float unit = pow2f(bad ? 0 : -ke);
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = bad ? 0.f : __uint_as_float(w[i] << 16) * unit;
            y[2 * i + 1] = bad ? 0.f : __uint_as_float(w[i] & 0xFFFF0000u) * unit;
        }
        uint8_t *blk = block_ptr(pool, page, id.head, id.is_v);
        if constexpr (FMT == NVFP4_KV_E4M3) {
            uint2 c;
            c.x = f32x2_to_e4m3x2(y[0], y[1]) | f32x2_to_e4m3x2(y[2], y[3]) << 16;
            c.y = f32x2_to_e4m3x2(y[4], y[5]) | f32x2_to_e4m3x2(y[6], y[7]) << 16;
            *reinterpret_cast<uint2 *>(blk + at * R::kCode + lane * 8) = c;
        } else {
            const uint32_t sb = bad ? 0u
                                    : f32_to_e4m3_satfinite(__fdiv_rn(__uint_as_float(block_max << 16), 6.f) * unit);
            const float s = e4m3_to_f32(sb);
            uint32_t c = 0;
            if (sb != 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    c |= f32x2_to_e2m1x2(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s)) << (8 * i);
            }
            *reinterpret_cast<uint32_t *>(blk + at * R::kCode + lane * 4) = c;
            if (lane % 2 == 0)
                blk[(R::kCode << pool.page_shift) + at * R::kScale + lane / 2] = (uint8_t)sb;
        }
        if (lane == 0)
            blk[((R::kCode + R::kScale) << pool.page_shift) + at] = (uint8_t)(bad ? kNanRow : (uint32_t)(ke + 127));
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(Pool pool, uint16_t *__restrict__ k, int64_t k_ld,
                                                        uint16_t *__restrict__ v, int64_t v_ld,
                                                        const int64_t *__restrict__ slots, uint32_t n_rows)
{
    constexpr int L = D / 8;
    using R = Row<FMT, D>;
    const int lane = threadIdx.x % L;
    const uint32_t per_grid = gridDim.x * (kThreads / L);
    for (uint32_t r = blockIdx.x * (kThreads / L) + threadIdx.x / L; r < n_rows;
         r = r + per_grid < r ? n_rows : r + per_grid) {
        const RowId id = row_id(r, pool.heads);
        const int64_t slot = slots[id.token];
        const int64_t page = slot >> pool.page_shift;
        uint4 out = make_uint4(0, 0, 0, 0);
        if (page >= pool.n_pages) {
            if (lane == 0)
                report(pool.status, kStatusKvReadSlot);
        } else if (slot >= 0) {
            const int at = (int)(slot & ((1 << pool.page_shift) - 1));
            const uint8_t *blk = block_ptr(pool, page, id.head, id.is_v);
            const float unit = exp2_byte(blk[((R::kCode + R::kScale) << pool.page_shift) + at]);
            uint32_t o[4];
            if constexpr (FMT == NVFP4_KV_E4M3) {
                const uint2 c = *reinterpret_cast<const uint2 *>(blk + at * R::kCode + lane * 8);
                const uint32_t two[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f16x2_to_f32(e4m3x2_to_f16x2((uint16_t)two[i]));
                    o[i] = f32x2_to_bf16x2(f.x * unit, f.y * unit);
                }
            } else {
                const uint32_t c = *reinterpret_cast<const uint32_t *>(blk + at * R::kCode + lane * 4);
                const float s = e4m3_to_f32(blk[(R::kCode << pool.page_shift) + at * R::kScale + lane / 2]) * unit;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f16x2_to_f32(e2m1x2_to_f16x2(c >> (8 * i) & 0xFFu));
                    o[i] = f32x2_to_bf16x2(f.x * s, f.y * s);
                }
            }
            out = make_uint4(o[0], o[1], o[2], o[3]);
        }
        uint16_t *dst = id.is_v ? v + (int64_t)id.token * v_ld : k + (int64_t)id.token * k_ld;
        *reinterpret_cast<uint4 *>(dst + (int64_t)id.head * D + lane * 8) = out;
    }
}

// Calls f(format, head_dim) with both as compile-time constants.
template <class F>
void by_format(const nvfp4_kv_cache *c, F &&f)
{
    using std::integral_constant;
    if (c->format == NVFP4_KV_E4M3)
        c->head_dim == 64 ? f(integral_constant<int, 0>{}, integral_constant<int, 64>{})
                          : f(integral_constant<int, 0>{}, integral_constant<int, 128>{});
    else
        c->head_dim == 64 ? f(integral_constant<int, 1>{}, integral_constant<int, 64>{})
                          : f(integral_constant<int, 1>{}, integral_constant<int, 128>{});
}

int check_rows(const nvfp4_kv_cache *c, const void *k, int64_t k_ld, const void *v, int64_t v_ld,
               const int64_t *slots, int64_t n_tokens)
{
    if (n_tokens < 0)
        return NVFP4_ERR_INVALID_ARG;
    if (n_tokens == 0)
        return NVFP4_OK;
    if (n_tokens >= (INT64_C(1) << 30) / c->n_kv_heads)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    const int64_t width = (int64_t)c->n_kv_heads * c->head_dim;
    if (k_ld < width || v_ld < width || k_ld % 8 != 0 || v_ld % 8 != 0 ||
        k_ld > (INT64_C(1) << 60) / n_tokens || v_ld > (INT64_C(1) << 60) / n_tokens)
        return NVFP4_ERR_INVALID_ARG;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
        return NVFP4_ERR_INVALID_ARG;
    return NVFP4_OK;
}

// One round of resident CTAs at most; each group of lanes strides over rows.
uint32_t row_grid(uint32_t n_rows, int head_dim)
{
    const uint32_t per_cta = kThreads / (head_dim / 8);
    const uint32_t need = (n_rows + per_cta - 1) / per_cta;
    return need < 152 * 8 ? need : 152 * 8;
}

}  // namespace

int make_pool(const nvfp4_kv_cache *c, void *workspace, size_t workspace_bytes, Pool *out)
{
    if (!c)
        return NVFP4_ERR_INVALID_ARG;
    const size_t page = nvfp4_kv_page_bytes(c->page_size, c->n_kv_heads, c->head_dim, c->format);
    if (page == 0)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (c->n_pages < 0 || c->n_pages > INT32_MAX)
        return NVFP4_ERR_INVALID_ARG;
    if (c->n_pages > 0 && (!c->pool || !aligned(c->pool, 16)))
        return NVFP4_ERR_INVALID_ARG;
    if (workspace && (!aligned(workspace, 16) || workspace_bytes < kKvWorkspaceBytes))
        return aligned(workspace, 16) ? NVFP4_ERR_WORKSPACE : NVFP4_ERR_INVALID_ARG;
    out->base = static_cast<uint8_t *>(c->pool);
    out->n_pages = c->n_pages;
    out->page_bytes = (int64_t)page;
    out->block_bytes = (int32_t)(page / (2 * (size_t)c->n_kv_heads));
    out->page_shift = 0;
    while ((1 << out->page_shift) < c->page_size)
        ++out->page_shift;
    out->heads = c->n_kv_heads;
    out->status = workspace ? reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + kStatusWordOffset)
                            : nullptr;
    return NVFP4_OK;
}

}  // namespace kv
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_kv_page_bytes(int32_t page_size, int32_t n_kv_heads, int32_t head_dim, int32_t format)
{
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0 || n_kv_heads < 1 ||
        n_kv_heads > 1024 || (head_dim != 64 && head_dim != 128) ||
        (format != NVFP4_KV_E4M3 && format != NVFP4_KV_NVFP4))
        return 0;
    const size_t row = format == NVFP4_KV_E4M3 ? head_dim + 1 : head_dim / 2 + head_dim / 16 + 1;
    return row * page_size * 2 * (size_t)n_kv_heads;
}

int nvfp4_kv_append(const nvfp4_kv_cache *cache, const uint16_t *k, int64_t k_ld, const uint16_t *v, int64_t v_ld,
                    const int64_t *slots, int64_t n_tokens, void *workspace, size_t workspace_bytes,
                    nvfp4_stream_t stream)
{
    kv::Pool pool;
    int rc = kv::make_pool(cache, workspace, workspace_bytes, &pool);
    if (rc == NVFP4_OK)
        rc = kv::check_rows(cache, k, k_ld, v, v_ld, slots, n_tokens);
    if (rc != NVFP4_OK || n_tokens == 0)
        return rc;
    const uint32_t rows = (uint32_t)(n_tokens * 2 * cache->n_kv_heads);
    const uint32_t grid = kv::row_grid(rows, cache->head_dim);
    kv::by_format(cache, [&](auto fmt, auto d) {
        kv::append_kernel<fmt.value, d.value>
            <<<grid, kv::kThreads, 0, (cudaStream_t)stream>>>(pool, k, k_ld, v, v_ld, slots, rows);
    });
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

int nvfp4_kv_read(const nvfp4_kv_cache *cache, uint16_t *k, int64_t k_ld, uint16_t *v, int64_t v_ld,
                  const int64_t *slots, int64_t n_tokens, void *workspace, size_t workspace_bytes,
                  nvfp4_stream_t stream)
{
    kv::Pool pool;
    int rc = kv::make_pool(cache, workspace, workspace_bytes, &pool);
    if (rc == NVFP4_OK)
        rc = kv::check_rows(cache, k, k_ld, v, v_ld, slots, n_tokens);
    if (rc != NVFP4_OK || n_tokens == 0)
        return rc;
    const uint32_t rows = (uint32_t)(n_tokens * 2 * cache->n_kv_heads);
    const uint32_t grid = kv::row_grid(rows, cache->head_dim);
    kv::by_format(cache, [&](auto fmt, auto d) {
        kv::read_kernel<fmt.value, d.value>
            <<<grid, kv::kThreads, 0, (cudaStream_t)stream>>>(pool, k, k_ld, v, v_ld, slots, rows);
    });
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // extern "C"
