// Short causal convolution per channel over packed sequences and for single tokens.
//
//   v[t][c] = bias[c] + sum_k w[c][k] x[t - W + 1 + k][c],  W = 2, 3 or 4 taps
//   y = v or v * sigmoid(v)
//
// 2W flops an element against 4 (16-bit) or 8 bytes: bound by memory. A thread takes 16 bytes of
// channels (at any alignment; a row's last ones may be fewer) and a run of 8 rows of one sequence,
// with the run's rows and the W - 1 rows before it in registers, so x is read once apart from the
// W - 1 rows at each run's start, which the neighbouring run has in the L2. All of a run's loads are
// issued before the first product. The thread with a sequence's first run also writes the
// sequence's new state: it is the only one that reads the old one, so nothing has to wait.
//
// Long runs read fewer rows twice, short ones put more loads in flight. In runs of 4, 8, 16 and 32 rows,
// 4 taps: 16384 x 4352 bfloat16 67, 54, 54 and 57 us (5.3 TB/s in runs of 8), 4096 x 4352 21.1, 16.6, 19.5
// and 23.4, 512 x 4352 5.2, 5.1, 6.9 and 10.9, 18848 x 384 float32 13.5, 12.6, 12.9 and 15.5 (4.6 TB/s).
// A large copy reaches 4.8 TB/s on the same card. New rows of a few sequences are bound by the launch.
#include "sequence_device.h"

namespace bl {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 8;  // rows of a thread

// channels: left of the row from c on, of which this vector takes at most V.
template <typename T, int V, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, int channels, float (&w)[V][W], float (&bias)[V]) {
    const int count = channels < V ? channels : V;
    const T *wp = static_cast<const T *>(a.weight) + static_cast<size_t>(c) * W;
    Vec<T, V> raw[W];  // the channels' taps as they lie, W after W
#pragma unroll
    for (int k = 0; k < W; ++k) raw[k] = load_vector<false, T, V>(wp + k * V, count * W - k * V);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[i][k] = static_cast<float>(raw[(i * W + k) / V][(i * W + k) % V]);
        bias[i] = 0.0f;
    }
    if (a.bias != nullptr) {
        const Vec<T, V> b = load_vector<false, T, V>(static_cast<const T *>(a.bias) + c, count);
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = static_cast<float>(b[i]);
    }
}

template <typename T, int V, int W, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void conv_kernel(ConvArgs a, unsigned vectors, unsigned long long threads) {
    using X = Vec<T, V>;
    const unsigned long long id = static_cast<unsigned long long>(workgroup_number()) * kThreads + threadIdx.x;
    if (id >= threads) return;
    const int run = static_cast<int>(id / vectors);
    const int c = static_cast<int>(id % vectors) * V;
    const int channels = a.channels - c;  // of this vector, at least V but for a row's last one
    auto load = [&](const T *p) { return load_vector<ALIGNED, T, V>(p, channels); };
    const int j = sequence_of_run(a.seq, run, kRun);
    const Span span = span_of(a.seq, j);
    const long long at = static_cast<long long>(run - run_base(a.seq, j, kRun)) * kRun;
    if (at < 0 || at >= span.length) return;
    const int place = a.state != nullptr ? place_of(a.seq, j) : 0;
    if (place < 0) return;
    const int offset = static_cast<int>(at);
    const int count = span.length - offset < kRun ? span.length - offset : kRun;

    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(span.first) * a.x_stride + c;
    T *y = static_cast<T *>(a.y) + static_cast<size_t>(span.first) * a.y_stride + c;
    T *state = a.state != nullptr
                   ? static_cast<T *>(a.state) + static_cast<size_t>(place) * (W - 1) * a.channels + c
                   : nullptr;

    X rows[kRun + W - 1];  // rows offset - (W - 1) .. offset + kRun - 1
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
        rows[W - 1 + r] = X{};
        if (r < count) rows[W - 1 + r] = load(x + static_cast<size_t>(offset + r) * a.x_stride);
    }
    if (offset == 0) {
        const bool kept = state != nullptr && !starts_fresh(a.seq, j);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            rows[r] = X{};
            if (kept) rows[r] = load(state + static_cast<size_t>(r) * a.channels);
        }
        if (state != nullptr) {
            // the last W - 1 rows of (old state, x): old rows while the sequence is shorter
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                const int from = span.length - (W - 1) + r;  // row of x; negative: kept row from + W - 1
                X v{};
                if (from >= 0) {
                    v = load(x + static_cast<size_t>(from) * a.x_stride);
                } else {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        if (k == from + W - 1) v = rows[k];
                }
                store_vector<ALIGNED, T, V>(state + static_cast<size_t>(r) * a.channels, v, channels);
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            // a run starts at a multiple of kRun >= W - 1, so these rows are the sequence's own
            rows[r] = load(x + static_cast<size_t>(offset - (W - 1) + r) * a.x_stride);
        }
    }
    static_assert(kRun >= W - 1, "a run's predecessors lie in the run before it");

    float w[V][W], bias[V];
    load_taps<T, V, W>(a, c, channels, w, bias);
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
        X out;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) v = fmaf(w[i][k], static_cast<float>(rows[r + k][i]), v);
            out[i] = static_cast<T>(a.silu ? silu<T>(v) : v);
        }
        if (r < count) store_vector<ALIGNED, T, V>(y + static_cast<size_t>(offset + r) * a.y_stride, out, channels);
    }
}

template <typename T, int V, int W, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(ConvArgs a, unsigned vectors, unsigned long long threads) {
    using X = Vec<T, V>;
    const unsigned long long id = static_cast<unsigned long long>(workgroup_number()) * kThreads + threadIdx.x;
    if (id >= threads) return;
    const int row = static_cast<int>(id / vectors);
    const int c = static_cast<int>(id % vectors) * V;
    const int channels = a.channels - c;
    auto load = [&](const T *p) { return load_vector<ALIGNED, T, V>(p, channels); };
    const int place = place_of(a.seq, row);
    if (place < 0) return;
    T *state = static_cast<T *>(a.state) + static_cast<size_t>(place) * (W - 1) * a.channels + c;
    X rows[W];
    rows[W - 1] = load(static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.x_stride + c);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) rows[r] = load(state + static_cast<size_t>(r) * a.channels);
    float w[V][W], bias[V];
    load_taps<T, V, W>(a, c, channels, w, bias);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        store_vector<ALIGNED, T, V>(state + static_cast<size_t>(r) * a.channels, rows[r + 1], channels);
    }
    X out;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float v = bias[i];
#pragma unroll
        for (int k = 0; k < W; ++k) v = fmaf(w[i][k], static_cast<float>(rows[k][i]), v);
        out[i] = static_cast<T>(a.silu ? silu<T>(v) : v);
    }
    store_vector<ALIGNED, T, V>(static_cast<T *>(a.y) + static_cast<size_t>(row) * a.y_stride + c, out, channels);
}

template <typename T, int W, bool ALIGNED>
hipError_t run_conv(const ConvArgs &a, bool step, hipStream_t stream) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const unsigned vectors = (static_cast<unsigned>(a.channels) + V - 1) / V;
    const unsigned long long runs =
        step ? static_cast<unsigned long long>(a.seq.rows)
             : static_cast<unsigned long long>(a.seq.rows) / kRun + static_cast<unsigned long long>(a.seq.sequences);
    const unsigned long long threads = runs * vectors;
    const unsigned long long blocks = (threads + kThreads - 1) / kThreads;
    if (blocks == 0) return hipSuccess;
    return launch(step ? conv_step_kernel<T, V, W, ALIGNED> : conv_kernel<T, V, W, ALIGNED>, blocks, kThreads, stream, a,
                  vectors, threads);
}

template <typename T, bool ALIGNED>
hipError_t by_taps(const ConvArgs &a, bool step, hipStream_t stream) {
    switch (a.taps) {
        case 2: return run_conv<T, 2, ALIGNED>(a, step, stream);
        case 3: return run_conv<T, 3, ALIGNED>(a, step, stream);
        case 4: return run_conv<T, 4, ALIGNED>(a, step, stream);
        default: return hipErrorInvalidValue;
    }
}

template <typename T>
hipError_t by_alignment(const ConvArgs &a, bool step, hipStream_t stream) {
    constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                           reinterpret_cast<uintptr_t>(a.state);
    // vectors at any element cost these 56, 18, 5.7 and 13.2 us in place of 54, 16.6, 5.1 and 12.6
    const bool wide = bits % 16 == 0 && a.channels % kVec == 0 && a.x_stride % kVec == 0 && a.y_stride % kVec == 0;
    return wide ? by_taps<T, true>(a, step, stream) : by_taps<T, false>(a, step, stream);
}

hipError_t by_type(const ConvArgs &a, Elem type, bool step, hipStream_t stream) {
    switch (type) {
        case Elem::f32: return by_alignment<float>(a, step, stream);
        case Elem::bf16: return by_alignment<__bf16>(a, step, stream);
        default: return by_alignment<_Float16>(a, step, stream);
    }
}

}  // namespace

hipError_t launch_conv(const ConvArgs &args, Elem type, hipStream_t stream) { return by_type(args, type, false, stream); }

hipError_t launch_conv_step(const ConvArgs &args, Elem type, hipStream_t stream) { return by_type(args, type, true, stream); }

}  // namespace bl
