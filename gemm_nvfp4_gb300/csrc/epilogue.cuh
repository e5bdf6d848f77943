// epilogue.cuh -- what the product kernels do with a sum before they store it, when a
// call asks for more than the sum (nvfp4_gemm_epilogue, nvfp4_fp6_gemm_epilogue):
//     y = residual + act(sum + bias), in fp32.
// The kernels take it as a template flag, so that the calls without one stay what they were.
//
// Little of it is overlapped with a product, so it is kept off the sums' way: the choice of the activation is made once
// for many values, quotients and exponentials are the short ones (a 5120 -> 17408 product of 509 tokens with bias and
// tanh GELU takes 81 us, as without; with the choice made for each value it took 134, with tanhf's accuracy 104), and
// a tile's residual and bias are asked into L2 while its product runs.
#pragma once

#include "../../include/nvfp4.h"
#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {

// sum * Phi(sum) for the erf form: normcdff has no cancellation in the lower tail;
// sum * sigmoid(2 u) for the tanh form, which is the same as (1 + tanh(u)) / 2 without its cancellation.
// NaN stays NaN (fmaxf would drop it).  The quotients are within two ulps (zero for divisors beyond 2^126, where they are
// below 2^-120); __expf is off by 2^-22 for each unit of its argument, which the bound for the tanh form allows for.
template <int ACT>
NVFP4_DEVINL float activate(float v)
{
    if (ACT == NVFP4_ACT_SILU)
        return __fdividef(v, 1.0f + expf(-v));
    if (ACT == NVFP4_ACT_GELU)
        return v * normcdff(v);
    if (ACT == NVFP4_ACT_GELU_TANH)
        return __fdividef(v, 1.0f + __expf(-1.5957691216057308f * fmaf(0.044715f * v * v, v, v)));
    if (ACT == NVFP4_ACT_RELU)
        return v < 0.f ? 0.f : v;
    if (ACT == NVFP4_ACT_RELU2)
        return v < 0.f ? 0.f : v * v;
    return v;
}

template <int ACT, int N>
NVFP4_DEVINL void activate_each(float (&v)[N], int n)
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (N <= 4 || j < n)
            v[j] = activate<ACT>(v[j]);
}

// The first n values.
template <int N>
NVFP4_DEVINL void activate_all(int act, float (&v)[N], int n = N)
{
    switch (act) {
    case NVFP4_ACT_SILU: activate_each<NVFP4_ACT_SILU>(v, n); break;
    case NVFP4_ACT_GELU: activate_each<NVFP4_ACT_GELU>(v, n); break;
    case NVFP4_ACT_GELU_TANH: activate_each<NVFP4_ACT_GELU_TANH>(v, n); break;
    case NVFP4_ACT_RELU: activate_each<NVFP4_ACT_RELU>(v, n); break;
    case NVFP4_ACT_RELU2: activate_each<NVFP4_ACT_RELU2>(v, n); break;
    default: break;
    }
}

NVFP4_DEVINL float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

NVFP4_DEVINL float epilogue_bias(const Epilogue &e, int64_t m)
{
    if (!e.bias)
        return 0.f;
    return e.bias_bf16 ? bf16_value(__ldg(static_cast<const uint16_t *>(e.bias) + m)) : __ldg(static_cast<const float *>(e.bias) + m);
}

// The residual of row m of tokens n0 .. n0 + N - 1 (below M and n_end), as it is stored: ordinary loads, whose memory may
// be the output's, and all before the first use.
template <int N>
NVFP4_DEVINL void load_residual(const Epilogue &e, uint32_t (&r)[N], int64_t n0, int64_t n_end, int64_t m, int64_t M)
{
    if (!e.residual || m >= M)
        return;
    const int64_t at = n0 * e.residual_ld + m;
    if (e.residual_bf16) {
        const uint16_t *p = static_cast<const uint16_t *>(e.residual) + at;
#pragma unroll
        for (int j = 0; j < N; ++j)
            r[j] = n0 + j < n_end ? p[j * e.residual_ld] : 0u;
    } else {
        const uint32_t *p = static_cast<const uint32_t *>(e.residual) + at;
#pragma unroll
        for (int j = 0; j < N; ++j)
            r[j] = n0 + j < n_end ? p[j * e.residual_ld] : 0u;
    }
}

template <int N>
NVFP4_DEVINL void add_residual(const Epilogue &e, float (&v)[N], const uint32_t (&r)[N])
{
    if (!e.residual)
        return;
#pragma unroll
    for (int j = 0; j < N; ++j)
        v[j] = __uint_as_float(e.residual_bf16 ? r[j] << 16 : r[j]) + v[j];
}

// Adds the residual of row m to the values of tokens n0 .. n0 + N - 1, below n_end: every load before the first use.
template <int N>
NVFP4_DEVINL void add_residual(const Epilogue &e, float (&v)[N], int64_t n0, int64_t n_end, int64_t m)
{
    if (!e.residual)
        return;
    const int64_t at = n0 * e.residual_ld + m;
    if (e.residual_bf16) {
        const uint16_t *p = static_cast<const uint16_t *>(e.residual) + at;
        uint16_t r[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            r[j] = n0 + j < n_end ? p[j * e.residual_ld] : (uint16_t)0;
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = bf16_value(r[j]) + v[j];
    } else {
        const float *p = static_cast<const float *>(e.residual) + at;
        float r[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            r[j] = n0 + j < n_end ? p[j * e.residual_ld] : 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = r[j] + v[j];
    }
}

// Output of row m, token n.
NVFP4_DEVINL float epilogue_value(const Epilogue &e, float sum, int64_t n, int64_t m)
{
    float v[1] = {sum + epilogue_bias(e, m)};
    activate_all(e.act, v);
    add_residual(e, v, n, n + 1, m);
    return v[0];
}

NVFP4_DEVINL void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Asks the residual of rows m0 .. m0 + n_rows - 1 (within M) of tokens n0 .. n_end - 1, and their bias, into L2: thread t
// of `threads` takes its share of the 128-byte lines.
NVFP4_DEVINL void epilogue_prefetch(const Epilogue &e, int64_t n0, int64_t n_end, int64_t m0, int n_rows, int64_t M, int t, int threads)
{
    n_rows = M - m0 < n_rows ? (int)(M - m0) : n_rows;
    if (n_rows <= 0)
        return;
    if (e.bias) {
        const int size = e.bias_bf16 ? 2 : 4;
        if (t * 128 < n_rows * size)
            prefetch_l2(static_cast<const uint8_t *>(e.bias) + m0 * size + t * 128);
    }
    if (e.residual) {
        const int size = e.residual_bf16 ? 2 : 4, lines = (n_rows * size + 127) / 128;
        const int total = (int)(n_end - n0) * lines;
        for (int i = t; i < total; i += threads) {
            const int n = i / lines;
            prefetch_l2(static_cast<const uint8_t *>(e.residual) + ((n0 + n) * e.residual_ld + m0) * size + (i - n * lines) * 128);
        }
    }
}

}  // namespace nvfp4
