// epilogue.cuh -- what the product kernels do with a sum before they store it, when a
// call asks for more than the sum (nvfp4_gemm_epilogue, nvfp4_fp6_gemm_epilogue):
//     y = residual + act(sum + bias), in fp32.
// The kernels take it as a template flag, so that the calls without one stay what they were.
#pragma once

#include "../../include/nvfp4.h"
#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {

// sum * Phi(sum) for the erf form: normcdff has no cancellation in the lower tail;
// sum * sigmoid(2 u) for the tanh form, which is the same as (1 + tanh(u)) / 2 without its cancellation.
// NaN stays NaN (fmaxf would drop it).
NVFP4_DEVINL float activate(int act, float v)
{
    switch (act) {
    case NVFP4_ACT_SILU: return __fdiv_rn(v, 1.0f + expf(-v));
    case NVFP4_ACT_GELU: return v * normcdff(v);
    case NVFP4_ACT_GELU_TANH: return __fdiv_rn(v, 1.0f + expf(-1.5957691216057308f * fmaf(0.044715f * v * v, v, v)));
    case NVFP4_ACT_RELU: return v < 0.f ? 0.f : v;
    case NVFP4_ACT_RELU2: return v < 0.f ? 0.f : v * v;
    default: return v;
    }
}

NVFP4_DEVINL float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

NVFP4_DEVINL float epilogue_bias(const Epilogue &e, int64_t m)
{
    if (!e.bias)
        return 0.f;
    return e.bias_bf16 ? bf16_value(__ldg(static_cast<const uint16_t *>(e.bias) + m)) : __ldg(static_cast<const float *>(e.bias) + m);
}

// (an ordinary load: the output may be the residual's own memory)
NVFP4_DEVINL float epilogue_residual(const Epilogue &e, int64_t n, int64_t m)
{
    if (!e.residual)
        return 0.f;
    const int64_t at = n * e.residual_ld + m;
    return e.residual_bf16 ? bf16_value(static_cast<const uint16_t *>(e.residual)[at]) : static_cast<const float *>(e.residual)[at];
}

// Output of row m, token n.
NVFP4_DEVINL float epilogue_value(const Epilogue &e, float sum, int64_t n, int64_t m)
{
    const float r = epilogue_residual(e, n, m);
    const float v = activate(e.act, sum + epilogue_bias(e, m));
    return e.residual ? r + v : v;
}

}  // namespace nvfp4
