// Device helpers shared by the kernels of the causal sequence operators.
#pragma once

#include <hip/hip_runtime.h>

#include "sequence_internal.h"

namespace bl {

// A grid's first dimension counts work-items in 32 bits and is cut short without an error beyond. Workgroups
// of a larger launch are numbered over two dimensions, kColumns in a row; the numbers of the last row may
// pass the count, which every kernel checks.
constexpr unsigned kColumns = 1u << 20;
constexpr unsigned long long kMostWorkgroups = (1ull << 31) - kColumns;  // so that every number fits an int

__device__ __forceinline__ unsigned workgroup_number() { return blockIdx.y * kColumns + blockIdx.x; }

template <class T>
struct AsIs {
    typedef T type;
};

// Starts a kernel of `blocks` workgroups, at most kMostWorkgroups, and returns what became of this launch: the
// thread's last error, which a launch by its own syntax leaves, may be an earlier call's.
template <class... Params>
hipError_t launch(void (*kernel)(Params...), unsigned long long blocks, unsigned threads, hipStream_t stream,
                  typename AsIs<Params>::type... params) {
    if (blocks > kMostWorkgroups) return hipErrorInvalidConfiguration;
    const bool narrow = blocks * threads <= 0xFFFFFFFFull;
    const dim3 grid(narrow ? static_cast<unsigned>(blocks) : kColumns,
                    narrow ? 1u : static_cast<unsigned>((blocks + kColumns - 1) / kColumns));
    void *values[] = {static_cast<void *>(&params)...};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, dim3(threads), values, 0, stream);
    if (e != hipSuccess) (void)hipGetLastError();  // it is returned
    return e;
}

template <typename T, int N>
using Vec = T __attribute__((ext_vector_type(N)));

// Global memory takes 16-byte accesses at any element's address; the compiler has to be told.
template <typename T, int N>
using AnyVec __attribute__((aligned(sizeof(T)))) = T __attribute__((ext_vector_type(N)));

// The N elements at p of which `count` exist. ALIGNED: all do, at a multiple of the vector's size.
template <bool ALIGNED, typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vector(const T *p, int count) {
    if constexpr (ALIGNED) {
        return *reinterpret_cast<const Vec<T, N> *>(p);
    } else {
        if (count >= N) return *reinterpret_cast<const AnyVec<T, N> *>(p);
        Vec<T, N> v = {};
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < count) v[i] = p[i];
        return v;
    }
}

template <bool ALIGNED, typename T, int N>
__device__ __forceinline__ void store_vector(T *p, const Vec<T, N> &v, int count) {
    if constexpr (ALIGNED) {
        *reinterpret_cast<Vec<T, N> *>(p) = v;
    } else if (count >= N) {
        *reinterpret_cast<AnyVec<T, N> *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < count) p[i] = v[i];
    }
}

template <typename T, int N>
__device__ __forceinline__ void load_floats(const T *p, float (&out)[N]) {
    const Vec<T, N> v = *reinterpret_cast<const Vec<T, N> *>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = static_cast<float>(v[i]);
}

template <typename T, int N>
__device__ __forceinline__ void store_floats(T *p, const float (&in)[N]) {
    Vec<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = static_cast<T>(in[i]);
    *reinterpret_cast<Vec<T, N> *>(p) = v;
}

// e^-v on v_exp_f32 (1 ulp; 0 below float32's normal range) with its exponent's rounding carried along:
// t + rest = -v log2 e, e^-v = 2^t (1 + rest ln 2). Where 2^t is 0 or infinite, rest may be neither.
__device__ __forceinline__ float exp_of_minus(float v) {
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.9259629911266175e-8f, kLn2 = 0.6931471805599453f;
    const float t = -kLog2e * v;
    const float e = __builtin_amdgcn_exp2f(t);
    const float rest = fmaf(-kLog2e, v, -t) - kLog2eLow * v;
    return e > 0.0f && e < __builtin_huge_valf() ? fmaf(e, rest * kLn2, e) : e;
}

// v * sigmoid(v), with v_rcp_f32 (1 ulp). For 16-bit tensors the exponent's rounding is dropped: |v| 2^-24
// of the value, far inside the output's rounding. A sigmoid below 2^-126, v < -87, counts as 0.
template <typename T>
__device__ __forceinline__ float silu(float v) {
    const float e = sizeof(T) == 4 ? exp_of_minus(v) : __builtin_amdgcn_exp2f(-1.4426950408889634f * v);
    return v * __builtin_amdgcn_rcpf(1.0f + e);
}

// One sequence's rows in a packed batch, cut to 0..rows.
struct Span {
    int first;
    int length;
};

__device__ __forceinline__ int clamp_row(int v, int rows) { return v < 0 ? 0 : (v > rows ? rows : v); }

__device__ __forceinline__ Span span_of(const SequenceArgs &s, int j) {
    const int first = clamp_row(s.starts[j], s.rows);
    const int end = clamp_row(s.starts[j + 1], s.rows);
    return {first, end > first ? end - first : 0};
}

// Runs of `size` rows that never cross a sequence: run r belongs to the last sequence j with
// starts[j] / size + j <= r, as its run r - (starts[j] / size + j). Sequence j has
// floor(starts[j + 1] / size) - floor(starts[j] / size) + 1 >= ceil(length / size) run numbers, so
// rows / size + sequences numbers cover every batch without a table of lengths; numbers past a
// sequence's end have no rows.
__device__ __forceinline__ int run_base(const SequenceArgs &s, int j, int size) {
    return clamp_row(s.starts[j], s.rows) / size + j;
}

__device__ __forceinline__ int sequence_of_run(const SequenceArgs &s, int run, int size) {
    int low = 0, high = s.sequences - 1;  // the answer is in low..high (run_base(0) may exceed run: then 0)
    while (low < high) {
        const int mid = (low + high + 1) >> 1;
        if (run_base(s, mid, size) <= run) {
            low = mid;
        } else {
            high = mid - 1;
        }
    }
    return low;
}

// The last sequence that passes, for a whole wave, where no sequence passes behind one that does not: 64
// places of the table at a time, so that 64 sequences take one load's time and 4096 take two. The
// first one is taken to pass.
template <class Passes>
__device__ __forceinline__ int last_sequence_wave(const SequenceArgs &s, const Passes &passes) {
    const int lane = threadIdx.x & 63;
    int low = 0, count = s.sequences;  // the answer is in low .. low + count - 1
    while (count > 1) {
        const int step = (count + 63) / 64;
        const int at = lane * step;  // lane 0 always passes: the answer is at low or behind it
        const bool ok = at < count && (lane == 0 || passes(low + at));
        const int ahead = (__popcll(__ballot(ok)) - 1) * step;
        low += ahead;
        count = count - ahead < step ? count - ahead : step;
    }
    return __builtin_amdgcn_readfirstlane(low);
}

// The same as sequence_of_run for a whole wave with one run.
__device__ __forceinline__ int sequence_of_run_wave(const SequenceArgs &s, int run, int size) {
    return last_sequence_wave(s, [&](int j) { return run_base(s, j, size) <= run; });
}

// The sequence with this row, for a whole wave.
__device__ __forceinline__ int sequence_of_row_wave(const SequenceArgs &s, int row) {
    return last_sequence_wave(s, [&](int j) { return clamp_row(s.starts[j], s.rows) <= row; });
}

// The cache place of sequence j: -1 for one that is padding.
__device__ __forceinline__ int place_of(const SequenceArgs &s, int j) {
    const int p = s.slots != nullptr ? s.slots[j] : j;
    return p >= 0 && p < s.places ? p : -1;
}

__device__ __forceinline__ bool starts_fresh(const SequenceArgs &s, int j) {
    return s.fresh != nullptr && s.fresh[j] != 0;
}

}  // namespace bl
