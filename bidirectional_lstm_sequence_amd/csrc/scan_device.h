// Device helpers shared by the two forms of the state space scan.
#pragma once

#include "sequence_device.h"

namespace bl {

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in [0, 1], and log1p(e) = 2 artanh(r) with
// r = e / (2 + e) <= 1/3: the series r + r^3/3 + ... to r^13/13 leaves 2^-26 of it. The quotient is
// v_rcp_f32's, put right by what it and the sum 2 + e left; the series' small part is added last. In a model
// of these steps with the units' 1 ulp the relative error is 6e-8 (rms) and 2.6e-7 at most from v = -20 to
// 10; log1p(exp) in float32 has 5.5e-8 and 2.8e-7.
__device__ __forceinline__ float softplus(float v) {
    const float e = exp_of_minus(fabsf(v));
    const float d = 2.0f + e, lost = e - (d - 2.0f);
    const float inverse = __builtin_amdgcn_rcpf(d);
    const float near = e * inverse;
    const float r = fmaf(fmaf(-near, d, e) - near * lost, inverse, near);
    const float q = r * r;
    float p = 1.0f / 13.0f;
    p = fmaf(p, q, 1.0f / 11.0f);
    p = fmaf(p, q, 1.0f / 9.0f);
    p = fmaf(p, q, 1.0f / 7.0f);
    p = fmaf(p, q, 1.0f / 5.0f);
    p = fmaf(p, q, 1.0f / 3.0f);
    return fmaf(2.0f * r, p * q, 2.0f * r) + fmaxf(v, 0.0f);
}

// The step D of a head from its element of dt and its bias.
__device__ __forceinline__ float step_from(float dt, float bias, bool through_softplus) {
    return through_softplus ? softplus(dt + bias) : dt + bias;
}

// The chunked form for element type T (scan_chunks.h); one source file instantiates each type.
template <typename T>
hipError_t launch_scan_chunks(const ScanArgs &args, int run_rows, hipStream_t stream);

}  // namespace bl
