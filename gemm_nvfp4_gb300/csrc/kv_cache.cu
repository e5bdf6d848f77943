// kv_cache.cu -- rows into and out of the quantised paged KV cache
// (nvfp4_kv_append, nvfp4_kv_read; the format is in include/nvfp4.h).
//
// Both are copies with a change of format, bound by HBM for many tokens (a
// 128-element bf16 row of 256 B becomes 129 or 73 B) and by the launch for
// few.  Measured on one GB300, 8 heads of 128: reading 65536 NVFP4 tokens back
// 55.8 us (6.2 TB/s, 0.91 of the measured copy bandwidth); append and read of
// 8192 NVFP4 tokens 19.4 us together (12.7 at that bandwidth), of one E4M3 token
// 3.5 us.  D / 8 neighbouring lanes hold one row, 8 elements (one 16-byte vector
// of bf16) each: loads and stores of values are whole 16-byte vectors, a row's
// maximum takes 3 or 4 shuffles, and an NVFP4 block of 16 is two lanes.
#include <cstdint>

#include "kernels.h"
#include "kv_layout.cuh"
#include "tcgen05.cuh"

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

// Rows of one pass of a group of lanes: their loads are all on their way before
// the first is used.
constexpr int kRowsAtOnce = 4;

// A group of lanes has one token and walks over its rows (K's heads, then V's),
// so that the slot is looked up once.  The groups of a CTA have consecutive
// tokens, which mostly lie in one page: together they touch whole runs of
// its codes, scales and exponents.  (With a token's heads side by side in a
// CTA instead, every 8 bytes of scales and byte of exponent cost a sector of
// their own, and reading 65536 NVFP4 tokens of 8 heads back took 98 us.)
// Few tokens are shared out by rows as well, `rows` of a token to a CTA.
struct RowWalk {
    uint32_t token;
    int begin, end;
};

template <int L>
NVFP4_DEVINL RowWalk row_walk(int heads, int rows)
{
    RowWalk w;
    w.token = blockIdx.x * (kThreads / L) + threadIdx.x / L;
    w.begin = (int)blockIdx.y * rows;
    w.end = min(w.begin + rows, 2 * heads);
    return w;
}

// A row's place in the pool; slot < 0 for a row that is left out.
struct Place {
    int64_t page;
    int at;
    bool there;
};

NVFP4_DEVINL Place place_of(const Pool &pool, int64_t slot, bool report_it, uint32_t code)
{
    Place p;
    p.page = slot >> pool.page_shift;
    p.at = (int)(slot & ((1 << pool.page_shift) - 1));
    p.there = slot >= 0 && p.page < pool.n_pages;
    if (slot >= 0 && !p.there && report_it)
        report_index(pool.status, code);
    return p;
}

// A quotient that is next rounded to a few bits, from a product with the
// reciprocal (off by less than 2^-21 of itself).  The roundings that follow, to
// E4M3 of a block's max / 6 and to E2M1 of an element / scale, have their ties at
// quotients of at most 5 bits, and the dividends (bf16 values times powers of two)
// have 8: a quotient that is not such a tie is off it by more than 2^-9 of
// itself.  So rounding the product to 12 bits makes every tie exact and moves no
// other quotient across one: the result is that of the rounded division.
NVFP4_DEVINL float quotient12(float x, float reciprocal)
{
    return __uint_as_float((__float_as_uint(x * reciprocal) + 0x800u) & ~0xFFFu);
}

NVFP4_DEVINL float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(Pool pool, const uint16_t *__restrict__ k, int64_t k_ld,
                                                          const uint16_t *__restrict__ v, int64_t v_ld,
                                                          const int64_t *__restrict__ slots, uint32_t n_tokens,
                                                          int rows)
{
    constexpr int L = D / 8, U = kRowsAtOnce;  // lanes of a row
    using R = Row<FMT, D>;
    const int lane = threadIdx.x % L;
    const uint32_t group_lanes = ((1u << L) - 1) << (threadIdx.x % 32 / L * L);
    const RowWalk w = row_walk<L>(pool.heads, rows);
    tc::griddep_launch_dependents();
    tc::griddep_wait();
    if (w.token >= n_tokens)
        return;
    const Place p = place_of(pool, slots[w.token], lane == 0, kStatusKvAppendSlot);
    if (!p.there)
        return;
    uint8_t *const page = block_ptr(pool, p.page, 0, 0);
    const uint16_t *const k_row = k + w.token * k_ld + lane * 8, *const v_row = v + w.token * v_ld + lane * 8;
    for (int j = w.begin; j < w.end; j += U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int head = j + u < pool.heads ? j + u : j + u - pool.heads;
            x[u] = make_uint4(0, 0, 0, 0);
            if (j + u < w.end)
                x[u] = ldg_v4((j + u < pool.heads ? k_row : v_row) + head * D);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= w.end)
                break;
            const int is_v = j + u >= pool.heads, head = j + u - (is_v ? pool.heads : 0);
            const uint32_t e[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            // maximum of the magnitudes as integers: NaN and infinity come out on top
            uint32_t m2 = __vmaxu2(__vmaxu2(e[0] & 0x7FFF7FFFu, e[1] & 0x7FFF7FFFu),
                                   __vmaxu2(e[2] & 0x7FFF7FFFu, e[3] & 0x7FFF7FFFu));
            uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
            m = max(m, __shfl_xor_sync(group_lanes, m, 1));
            const uint32_t block_max = m;  // of this lane pair's 16 elements
#pragma unroll
            for (int o = 2; o < L; o *= 2)
                m = max(m, __shfl_xor_sync(group_lanes, m, o));
            int ke = row_exponent<FMT>(__uint_as_float(m << 16));
            const bool bad = m >= 0x7F80u || ke > kExpMax;
            const float unit = pow2f(bad ? 0 : -ke);
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t two = bad ? 0u : e[i];
                y[2 * i] = __uint_as_float(two << 16) * unit;
                y[2 * i + 1] = __uint_as_float(two & 0xFFFF0000u) * unit;
            }
            uint8_t *blk = page + (int64_t)(head * 2 + is_v) * pool.block_bytes;
            if constexpr (FMT == NVFP4_KV_E4M3) {
                uint2 c;
                c.x = f32x2_to_e4m3x2(y[0], y[1]) | f32x2_to_e4m3x2(y[2], y[3]) << 16;
                c.y = f32x2_to_e4m3x2(y[4], y[5]) | f32x2_to_e4m3x2(y[6], y[7]) << 16;
                *reinterpret_cast<uint2 *>(blk + p.at * R::kCode + lane * 8) = c;
            } else {
                const uint32_t sb =
                    bad ? 0u : f32_to_e4m3_satfinite(quotient12(__uint_as_float(block_max << 16) * unit, 1.f / 6.f));
                uint32_t c = 0;
                if (sb != 0) {
                    const float r = rcp(e4m3_to_f32(sb));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        c |= f32x2_to_e2m1x2(quotient12(y[2 * i], r), quotient12(y[2 * i + 1], r)) << (8 * i);
                }
                *reinterpret_cast<uint32_t *>(blk + p.at * R::kCode + lane * 4) = c;
                if (lane % 2 == 0)
                    blk[(R::kCode << pool.page_shift) + p.at * R::kScale + lane / 2] = (uint8_t)sb;
            }
            if (lane == 0)
                blk[((R::kCode + R::kScale) << pool.page_shift) + p.at] =
                    (uint8_t)(bad ? kNanRow : (uint32_t)(ke + 127));
        }
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(Pool pool, uint16_t *__restrict__ k, int64_t k_ld,
                                                        uint16_t *__restrict__ v, int64_t v_ld,
                                                        const int64_t *__restrict__ slots, uint32_t n_tokens, int rows)
{
    constexpr int L = D / 8, U = kRowsAtOnce;
    using R = Row<FMT, D>;
    const int lane = threadIdx.x % L;
    const RowWalk w = row_walk<L>(pool.heads, rows);
    tc::griddep_launch_dependents();
    tc::griddep_wait();
    if (w.token >= n_tokens)
        return;
    const Place p = place_of(pool, slots[w.token], lane == 0, kStatusKvReadSlot);
    const uint8_t *const page = block_ptr(pool, p.there ? p.page : 0, 0, 0);
    uint16_t *const k_row = k + w.token * k_ld + lane * 8, *const v_row = v + w.token * v_ld + lane * 8;
    for (int j = w.begin; j < w.end; j += U) {
        uint2 code[U];
        uint32_t exps[U], scale[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            code[u] = make_uint2(0, 0);
            exps[u] = 127;
            scale[u] = 0;
            if (p.there && j + u < w.end) {
                const int is_v = j + u >= pool.heads, head = j + u - (is_v ? pool.heads : 0);
                const uint8_t *blk = page + (int64_t)(head * 2 + is_v) * pool.block_bytes;
                exps[u] = blk[((R::kCode + R::kScale) << pool.page_shift) + p.at];
                if constexpr (FMT == NVFP4_KV_E4M3) {
                    code[u] = *reinterpret_cast<const uint2 *>(blk + p.at * R::kCode + lane * 8);
                } else {
                    code[u].x = *reinterpret_cast<const uint32_t *>(blk + p.at * R::kCode + lane * 4);
                    scale[u] = blk[(R::kCode << pool.page_shift) + p.at * R::kScale + lane / 2];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= w.end)
                break;
            uint32_t o[4];
            const float unit = exp2_byte(exps[u]);
            if constexpr (FMT == NVFP4_KV_E4M3) {
                const uint32_t two[4] = {code[u].x & 0xFFFFu, code[u].x >> 16, code[u].y & 0xFFFFu, code[u].y >> 16};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f16x2_to_f32(e4m3x2_to_f16x2((uint16_t)two[i]));
                    o[i] = f32x2_to_bf16x2(f.x * unit, f.y * unit);
                }
            } else {
                const float s = e4m3_to_f32(scale[u]) * unit;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f16x2_to_f32(e2m1x2_to_f16x2(code[u].x >> (8 * i) & 0xFFu));
                    o[i] = f32x2_to_bf16x2(f.x * s, f.y * s);
                }
            }
            const int is_v = j + u >= pool.heads;
            *reinterpret_cast<uint4 *>((is_v ? v_row : k_row) + (j + u - (is_v ? pool.heads : 0)) * D) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
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

// Grid for n_tokens, and the rows of a token that a CTA walks over: all, unless
// that leaves fewer than 12 CTAs an SM.  (Append and read of 8192 NVFP4 tokens of
// 8 heads: 30.2 us with at least 4 an SM, 20.0 with 8, 19.4 with 12, 20.8 with 24.)
dim3 row_grid(uint32_t n_tokens, const nvfp4_kv_cache *c, int *rows)
{
    const uint32_t per_cta = kThreads / (c->head_dim / 8), all = 2 * c->n_kv_heads;
    const uint32_t ctas = (n_tokens + per_cta - 1) / per_cta;
    const uint32_t parts = ctas >= 152 * 12 ? 1 : 152 * 12 / ctas;
    *rows = (int)(parts >= all ? 1 : (all + parts - 1) / parts);
    return dim3(ctas, (all + *rows - 1) / *rows);
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
    int rows = 0;
    const dim3 grid = kv::row_grid((uint32_t)n_tokens, cache, &rows);
    cudaError_t e = cudaSuccess;
    kv::by_format(cache, [&](auto fmt, auto d) {
        e = launch_dependent(kv::append_kernel<fmt.value, d.value>, grid, kv::kThreads, 0, (cudaStream_t)stream, pool, k,
                             k_ld, v, v_ld, slots, (uint32_t)n_tokens, rows);
    });
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
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
    int rows = 0;
    const dim3 grid = kv::row_grid((uint32_t)n_tokens, cache, &rows);
    cudaError_t e = cudaSuccess;
    kv::by_format(cache, [&](auto fmt, auto d) {
        e = launch_dependent(kv::read_kernel<fmt.value, d.value>, grid, kv::kThreads, 0, (cudaStream_t)stream, pool, k, k_ld,
                             v, v_ld, slots, (uint32_t)n_tokens, rows);
    });
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // extern "C"
