// Selective state space scan over packed sequences and for single tokens.
//
//   D_t = softplus(dt_t + bias);  S_t = exp(D_t a) S_{t-1} + D_t x_t (x) b_t;  y_t = S_t c_t + d x_t
//
// per head, with a state S of [width][states] in float32, optionally y * z sigmoid(z). Two forms:
// single tokens (here) and packed sequences in chunks of rows (scan_chunks.h). A single row of a packed
// sequence is a chunk of one row there: walking over a packed sequence's rows one by one took 17 us
// against 34 for 512 single rows of 4 float32 heads of 64 channels and 64 states, but 99 against 52 for 64
// sequences of 4 rows of 32 bfloat16 heads of 64 channels and 256 states, and about a microsecond a row
// for one long sequence among many short ones, which the host cannot see.
#include "scan_device.h"

namespace bl {
namespace {

constexpr int kThreads = 256;

// One new row a sequence, bound by the state's bytes: a workgroup takes kThreads / (N / 4) * PASSES
// state rows of one head of one sequence, four states of a state row a lane, and loads all of a lane's
// state before it is used. 256 sequences of 64 heads of 64 channels and 128 states (1.08 GB of state
// moved) take 210 us, 5.1 TB/s; one takes 4 us.
template <typename T, int N, int PASSES>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(ScanArgs a, int parts) {
    constexpr int kLanes = N / 4;
    constexpr int kStep = kThreads / kLanes;  // state rows of one pass
    const int lane = threadIdx.x % kLanes;
    const unsigned number = workgroup_number();
    const int part = static_cast<int>(number % static_cast<unsigned>(parts));
    const int h = static_cast<int>(number / static_cast<unsigned>(parts) % static_cast<unsigned>(a.heads));
    const int row = static_cast<int>(number / static_cast<unsigned>(parts) / static_cast<unsigned>(a.heads));
    if (row >= a.seq.rows) return;
    const int place = place_of(a.seq, row);
    if (place < 0) return;
    const int g = h / (a.heads / a.groups);
    const int p0 = part * kStep * PASSES + threadIdx.x / kLanes;
    float *state = a.state + (static_cast<size_t>(place) * a.heads + h) * a.width * N + lane * 4;
    float s[PASSES][4];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int p = p0 + i * kStep;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = 0.0f;
        if (p < a.width) load_floats<float, 4>(state + static_cast<size_t>(p) * N, s[i]);
    }
    const float skip = a.d != nullptr ? a.d[h] : 0.0f;
    const float bias = a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f;
    float b[4], c[4];
    const T *bp = static_cast<const T *>(a.b) + row * a.b_stride + g * N + lane * 4;
    const T *cp = static_cast<const T *>(a.c) + row * a.c_stride + g * N + lane * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        b[e] = static_cast<float>(bp[e]);
        c[e] = static_cast<float>(cp[e]);
    }
    const float step = step_from(static_cast<float>(static_cast<const T *>(a.dt)[row * a.dt_stride + h]), bias, a.softplus);
    const float keep = expf(step * a.a[h]);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int p = p0 + i * kStep;
        const bool live = p < a.width;
        const float x = live ? static_cast<float>(static_cast<const T *>(a.x)[row * a.x_stride + h * a.width + p]) : 0.0f;
        const float in = step * x;
        float y = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] = fmaf(s[i][e], keep, in * b[e]);
            y = fmaf(s[i][e], c[e], y);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) y += __shfl_xor(y, o);
        if (lane == 0 && live) {
            y = fmaf(skip, x, y);
            if (a.z != nullptr) {
                y *= silu<T>(static_cast<float>(static_cast<const T *>(a.z)[row * a.z_stride + h * a.width + p]));
            }
            static_cast<T *>(a.y)[row * a.y_stride + h * a.width + p] = static_cast<T>(y);
        }
        if (live) store_floats<float, 4>(state + static_cast<size_t>(p) * N, s[i]);
    }
}

template <typename T, int N, int PASSES>
hipError_t run_step(const ScanArgs &a, hipStream_t stream) {
    constexpr int kStep = kThreads / (N / 4) * PASSES;
    const int parts = (a.width + kStep - 1) / kStep;
    const unsigned long long blocks =
        static_cast<unsigned long long>(a.seq.sequences) * static_cast<unsigned>(a.heads) * static_cast<unsigned>(parts);
    return launch(scan_step_kernel<T, N, PASSES>, blocks, kThreads, stream, a, parts);
}

// More passes keep more loads in flight and read b and c less often, fewer leave more workgroups: the
// most that leave two workgroups a CU. Single tokens of 64 bfloat16 heads of 64 channels and 128 states
// with 1, 2, 4 and 8 passes: 128 sequences 124, 93, 83 and 88 us, 8 sequences 11.9, 8.8, 8.0 and 8.9, one
// 3.6, 3.7, 4.5 and 6.1; 64 of 4 float32 heads of 64 channels and 64 states 4.7, 4.3 and 4.8 with 1, 2, 4.
template <typename T, int N>
hipError_t by_passes(const ScanArgs &a, hipStream_t stream) {
    constexpr long long kStep = kThreads / (N / 4);
    const long long most = static_cast<long long>(a.seq.sequences) * a.heads * ((a.width + kStep - 1) / kStep) / 512;
    if (most >= 4 && a.width >= 4 * kStep) return run_step<T, N, 4>(a, stream);
    if (most >= 2 && a.width >= 2 * kStep) return run_step<T, N, 2>(a, stream);
    return run_step<T, N, 1>(a, stream);
}

template <typename T>
hipError_t by_states(const ScanArgs &a, hipStream_t stream) {
    switch (a.states) {
        case 16: return by_passes<T, 16>(a, stream);
        case 32: return by_passes<T, 32>(a, stream);
        case 64: return by_passes<T, 64>(a, stream);
        case 128: return by_passes<T, 128>(a, stream);
        case 256: return by_passes<T, 256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

// Most rows of a run of the chunked form; more than `rows` = whole sequences. The lengths of the sequences
// are on the device, so the rule goes by their sum and number.
//  * Splitting costs the end states of most runs (the products with x and b a second time) and two
//    launches; it pays while whole sequences leave the chip's 512 places (two workgroups a CU) empty, or
//    one long sequence outlives the others. Measured with 64 heads of 64 channels and 128 states: one
//    sequence of 4096 rows 126, 99, 89, 110, 97 and 121 us in runs of 96, 192, 256, 384, 512 and 768 rows,
//    446 us whole; 24 unequal ones of 16384 rows together (the mean of 12 such batches) 324, 298, 287, 291,
//    295 and 313 us in runs of at most 256, 384, 512, 640, 768 and 1024. 4 float32 heads of 64 channels and
//    64 states, 32 sequences of 589 rows: 71, 63, 55, 62, 59, 76 and 77 us in runs of 32, 64, 96, 128, 256, 384
//    and 512, 92 us whole. The least run is where one sequence of 600 rows of the 64 heads is fastest: 50, 40,
//    38, 39 and 42 us in runs of 32, 64, 96, 128 and 160; fewer workgroups would take shorter ones, as 1500 rows
//    of the 4 heads 26, 28, 34 and 40 in runs of 32, 64, 96 and 128.
//  * With four times as many workgroups as places only a sequence of over twice the mean is split. Unequal
//    sequences of the 64 heads with and without this: 128 of 131072 rows together 1725 and 1924 us, 64 of 65536
//    936 and 977, 256 of 65536 978 and 979, but 64 of 32768 509 and 503, 512 of 131072 1950 and 1906.
int run_rows_of(const ScanArgs &a) {
    constexpr long long kPlaces = 512, kLeast = 96, kMost = 768;
    constexpr int kChannels = 128;  // of a workgroup
    const long long rows = a.seq.rows, sequences = a.seq.sequences;
    const long long blocks = a.groups * ((a.heads / a.groups * static_cast<long long>(a.width) + kChannels - 1) / kChannels);
    long long run = rows * blocks / kPlaces;
    run = run < kLeast ? kLeast : (run > kMost ? kMost : run);
    if (sequences * blocks >= 4 * kPlaces && run < 2 * rows / sequences) run = 2 * rows / sequences;
    run = (run + 31) / 32 * 32;
    return run >= rows ? 0x7FFFFFFF : static_cast<int>(run);
}

}  // namespace

size_t scan_scratch_bytes(const ScanArgs &a) {
    if (a.seq.rows == 0 || a.seq.sequences == 0) return 0;
    const int run = run_rows_of(a);
    if (run > a.seq.rows) return 0;
    // slots_of: of the later runs, of the first ones; the decays
    const size_t blocks = static_cast<size_t>(a.seq.rows / run);
    const size_t first = static_cast<size_t>(a.seq.sequences) <= blocks ? a.seq.sequences : blocks + 1;
    return ((blocks + first) * a.width * a.states + blocks) * a.heads * sizeof(float);
}

hipError_t launch_scan(const ScanArgs &a, Elem type, hipStream_t stream) {
    const int run = run_rows_of(a);
    switch (type) {
        case Elem::f32: return launch_scan_chunks<float>(a, run, stream);
        case Elem::bf16: return launch_scan_chunks<__bf16>(a, run, stream);
        default: return launch_scan_chunks<_Float16>(a, run, stream);
    }
}

hipError_t launch_scan_step(const ScanArgs &a, Elem type, hipStream_t stream) {
    switch (type) {
        case Elem::f32: return by_states<float>(a, stream);
        case Elem::bf16: return by_states<__bf16>(a, stream);
        default: return by_states<_Float16>(a, stream);
    }
}

}  // namespace bl
