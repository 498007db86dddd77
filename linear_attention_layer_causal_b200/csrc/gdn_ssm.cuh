// gdn_ssm.cuh -- pieces shared by the prefill and the decode of the selective
// state-space mixer.
#pragma once

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {

// Four activations as floats: 8 bytes of bf16 or 16 of float32.
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }

// The step length of one head and token: clamp(softplus(dt + bias)).  expf,
// not __expf: log-decays are sums of up to thousands of these, and there are
// only H of them per token.
__device__ __forceinline__ float ssm_delta(float dt, float bias, float lo, float hi) {
    const float x = dt + bias;
    const float sp = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
    return x != x ? x : fminf(fmaxf(sp, lo), hi); // NaN stays NaN
}

} // namespace gdn
