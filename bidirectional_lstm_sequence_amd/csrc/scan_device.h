// Device helpers shared by the two forms of the state space scan.
#pragma once

#include "sequence_device.h"

namespace bl {

__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }

// The step D of a head from its element of dt.
__device__ __forceinline__ float step_from(const ScanArgs &a, float dt, int h) {
    if (a.dt_bias != nullptr) dt += a.dt_bias[h];
    return a.softplus ? softplus(dt) : dt;
}

template <typename T>
__device__ __forceinline__ float load_dt(const ScanArgs &a, long long row, int h) {
    return static_cast<float>(static_cast<const T *>(a.dt)[row * a.dt_stride + h]);
}

// The chunked form for element type T (scan_chunks.h); one source file instantiates each type.
template <typename T>
hipError_t launch_scan_chunks(const ScanArgs &args, int run_rows, hipStream_t stream);

}  // namespace bl
