// Device helpers shared by the two forms of the state space scan.
#pragma once

#include "sequence_device.h"

namespace bl {

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in (0, 1], and log1p(e) = 2 artanh(r) with
// r = e / (2 + e) <= 1/3: the series r + r^3/3 + ... to r^13/13 leaves 2^-26 of it.
__device__ __forceinline__ float softplus(float v) {
    const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(v));
    const float r = e * __builtin_amdgcn_rcpf(2.0f + e);
    const float q = r * r;
    float p = 1.0f / 13.0f;
    p = fmaf(p, q, 1.0f / 11.0f);
    p = fmaf(p, q, 1.0f / 9.0f);
    p = fmaf(p, q, 1.0f / 7.0f);
    p = fmaf(p, q, 1.0f / 5.0f);
    p = fmaf(p, q, 1.0f / 3.0f);
    p = fmaf(p, q, 1.0f);
    return fmaf(2.0f * r, p, fmaxf(v, 0.0f));
}

// The step D of a head from its element of dt and its bias.
__device__ __forceinline__ float step_from(float dt, float bias, bool through_softplus) {
    return through_softplus ? softplus(dt + bias) : dt + bias;
}

// The chunked form for element type T (scan_chunks.h); one source file instantiates each type.
template <typename T>
hipError_t launch_scan_chunks(const ScanArgs &args, int run_rows, hipStream_t stream);

}  // namespace bl
