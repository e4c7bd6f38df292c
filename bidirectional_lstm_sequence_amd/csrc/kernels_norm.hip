// Root-mean-square norm of rows with the residual's addition and an output in 8 bits.
//
//   s = x + residual;  r = 1 / sqrt(mean(s^2) + eps);  y = s r w;  scale = max|y| / top;  q = y / scale
//
// About 20 flops an element, a division among them, against 3 to 16 bytes: bound by memory. A group of
// lanes takes a row and keeps it in registers, so every input is read once and every output written once:
// the sum of squares comes out of a first pass over them, y and max|y| out of a second, the codes out of
// a third. Scales and codes are those of the float32 y itself, so max|y| has a reduction of its own. Rows
// that no register file holds (BLOCKS = 0) are read a second time for y and in 8 bits a third, from the
// L2 where they fit. The sum s is not rounded to the tensor's type before it is normed.
//
// 8192 x 5120 rows with a residual to e4m3 or int8 take 56 us in bfloat16 (7 bytes an element), 5.2 TB/s, 58 in
// float16 and 107 in float32 (13 bytes), where a large copy reaches 4.8; 18848 x 256 float32 rows with a
// residual 14 us, 5.5 TB/s, partly from caches.
#include "sequence_device.h"

namespace bl {
namespace {

constexpr float kLeastScale = 0x1p-100f;
constexpr float kLeastEps = 0x1p-100f;  // beside it the squares of a row that float32 does not hold are nothing

// A sum or maximum over the lanes of a group: 64 (a wave) or a whole workgroup. Each CALL of a kernel has
// its own place for the waves' parts, so none has to wait until the last one's have been read.
template <int GROUP, int CALL, class Op>
__device__ __forceinline__ float over_group(float v, Op op) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = op(v, __shfl_xor(v, o));
    if constexpr (GROUP > 64) {
        __shared__ float parts[GROUP / 64];
        if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = v;
        __syncthreads();
        v = parts[0];
#pragma unroll
        for (int w = 1; w < GROUP / 64; ++w) v = op(v, parts[w]);
    }
    return v;
}

// y / scale rounded as a division does, from the rounded reciprocal: after one correction by what is left of
// y the quotient is off by less than a step of float32, and from there another one rounds it correctly
// (Markstein). Half of a division's instructions: 81920 rows of 256 bfloat16 to e4m3 37.0 us, 40.3 with those.
__device__ __forceinline__ float quotient(float y, float scale, float inverse) {
    float q = y * inverse;
    q = fmaf(fmaf(-q, scale, y), inverse, q);
    return fmaf(fmaf(-q, scale, y), inverse, q);
}

// V values of y as 8-bit codes of the quotients y / scale.
// e4m3: v_cvt_pk_fp8_f32 rounds to nearest even (OCP e4m3 on gfx950); the clamp keeps a quotient that
// rounding left just above the top inside the range.
template <bool ALIGNED, int V, Eight E>
__device__ __forceinline__ void store_eight(unsigned char *p, const float (&y)[V], float scale, int count) {
    const float inverse = 1.0f / scale;
    unsigned char code[V];
    if constexpr (E == Eight::e4m3) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float u = fminf(fmaxf(quotient(y[i], scale, inverse), -448.0f), 448.0f);
            const float v = fminf(fmaxf(quotient(y[i + 1], scale, inverse), -448.0f), 448.0f);
            const int two = __builtin_amdgcn_cvt_pk_fp8_f32(u, v, 0, false);
            code[i] = static_cast<unsigned char>(two);
            code[i + 1] = static_cast<unsigned char>(two >> 8);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            code[i] = static_cast<unsigned char>(
                static_cast<int>(rintf(fminf(fmaxf(quotient(y[i], scale, inverse), -127.0f), 127.0f))));
        }
    }
    Vec<unsigned char, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = code[i];
    store_vector<ALIGNED, unsigned char, V>(p, v, count);
}

// GROUP lanes a row, BLOCKS vectors of 16 bytes a lane in registers; BLOCKS = 0: any width, the row is
// read again for y and for the codes. ALIGNED: rows and width are multiples of a vector; else vectors lie at
// any element and a row's last one may be short.
template <typename T, bool ALIGNED, int GROUP, int BLOCKS, Eight E>
__global__ __launch_bounds__(GROUP < 256 ? 256 : GROUP) void norm_kernel(NormArgs a) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    constexpr int kThreads = GROUP < 256 ? 256 : GROUP;
    constexpr int kRows = kThreads / GROUP;
    const int lane = threadIdx.x % GROUP;
    const long long row = static_cast<long long>(workgroup_number()) * kRows + threadIdx.x / GROUP;
    if (row >= a.rows) return;  // whole waves (GROUP = 64) or no workgroup at all: no barrier is left behind
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const T *residual = a.residual != nullptr ? static_cast<const T *>(a.residual) + row * a.residual_stride : nullptr;
    const T *weight = static_cast<const T *>(a.weight);
    T *residual_out = a.residual_out != nullptr ? static_cast<T *>(a.residual_out) + row * a.residual_out_stride : nullptr;
    T *y = a.y != nullptr ? static_cast<T *>(a.y) + row * a.y_stride : nullptr;
    unsigned char *q = a.q + row * a.q_stride;

    auto floats = [&](const T *p, int c, float (&out)[V]) {
        const Vec<T, V> v = load_vector<ALIGNED, T, V>(p + c, a.width - c);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = static_cast<float>(v[i]);
    };
    auto store = [&](T *p, int c, const float (&in)[V]) {
        Vec<T, V> v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = static_cast<T>(in[i]);
        store_vector<ALIGNED, T, V>(p + c, v, a.width - c);
    };
    auto load = [&](int c, float (&s)[V]) {
        floats(x, c, s);
        if (residual != nullptr) {
            float r[V];
            floats(residual, c, r);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] += r[i];
        }
    };
    float sum = 0.0f, r = 0.0f, up = 1.0f, most = 0.0f, scale = 1.0f;
    auto measure = [&](const float (&s)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum = fmaf(s[i] * up, s[i] * up, sum);
    };
    auto settle = [&](const auto &measure_row) {
        auto add = [](float u, float v) { return u + v; };
        sum = over_group<GROUP, 0>(sum, add);
        // Without an eps to speak of, squares that left float32's range below count: the row's values are
        // measured again, times 2^100 (whose sum stays below 2^120), and are normed with it.
        double eps = a.eps;
        if (a.eps < kLeastEps && sum < 0x1p-80f) {
            up = 0x1p100f;
            eps *= 0x1p200;
            sum = 0.0f;
            measure_row();
            sum = over_group<GROUP, 2>(sum, add);
        }
        // in 64 bits, so that r is rounded once: v_rsq_f64's 2^-24 or better and one step of Newton's method,
        // 14.5 us for 18848 x 256 float32 rows where a square root and divisions take 15.0. A row of zeros
        // without an eps stays one, an infinite sum gives 0.
        const double mean = fma(static_cast<double>(sum), a.inverse_width, eps);
        double root = __builtin_amdgcn_rsq(mean);
        if (mean < __builtin_huge_val()) root *= fma(-0.5 * mean * root, root, 1.5);
        r = mean == 0.0 ? 0.0f : static_cast<float>(root);
    };
    auto norm = [&](int c, float (&s)[V]) {
        float w[V];
        floats(weight, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = s[i] * up * r * w[i];
            if constexpr (E != Eight::none) most = __builtin_elementwise_maximum(most, fabsf(s[i]));  // a NaN stays
        }
    };
    auto settle_scale = [&] {
        if constexpr (E != Eight::none) {
            constexpr float kTop = E == Eight::e4m3 ? 448.0f : 127.0f;
            most = over_group<GROUP, 1>(most, [](float u, float v) { return __builtin_elementwise_maximum(u, v); });
            const bool number = sum < __builtin_huge_valf() && most < __builtin_huge_valf();
            scale = most == 0.0f ? 1.0f : most / kTop;
            if (scale < kLeastScale) scale = kLeastScale;  // quotients of it stay finite
            if (!number) scale = __builtin_nanf("");
            if (lane == 0) a.scales[row] = scale;
        }
    };
    auto emit = [&](int c, const float (&y_row)[V]) {
        if (y != nullptr) store(y, c, y_row);
        if constexpr (E != Eight::none) store_eight<ALIGNED, V, E>(q + c, y_row, scale, a.width - c);
    };

    if constexpr (BLOCKS > 0) {
        float s[BLOCKS][V];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const int c = (b * GROUP + lane) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) s[b][i] = 0.0f;
            if (c < a.width) load(c, s[b]);
        }
        auto measure_row = [&] {
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) measure(s[b]);
        };
        measure_row();
        settle(measure_row);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const int c = (b * GROUP + lane) * V;
            if (c >= a.width) continue;
            if (residual_out != nullptr) store(residual_out, c, s[b]);
            norm(c, s[b]);
            if constexpr (E == Eight::none) emit(c, s[b]);
        }
        if constexpr (E != Eight::none) {
            settle_scale();
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const int c = (b * GROUP + lane) * V;
                if (c < a.width) emit(c, s[b]);
            }
        }
    } else {
        // outputs may be the inputs' own memory: nothing is written before a lane's last look,
        // and a lane reads only what it writes itself
        float s[V];
        auto measure_row = [&] {
            for (int c = lane * V; c < a.width; c += GROUP * V) {
                load(c, s);
                measure(s);
            }
        };
        measure_row();
        settle(measure_row);
        if constexpr (E != Eight::none) {
            for (int c = lane * V; c < a.width; c += GROUP * V) {
                load(c, s);
                norm(c, s);
            }
            settle_scale();
        }
        for (int c = lane * V; c < a.width; c += GROUP * V) {
            load(c, s);
            if (residual_out != nullptr) store(residual_out, c, s);
            norm(c, s);
            emit(c, s);
        }
    }
}

template <typename T, bool ALIGNED, int GROUP, int BLOCKS>
hipError_t run(const NormArgs &a, Eight eight, hipStream_t stream) {
    constexpr int kThreads = GROUP < 256 ? 256 : GROUP;
    constexpr int kRows = kThreads / GROUP;
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.rows) + kRows - 1) / kRows);
    switch (eight) {
        case Eight::none: return launch(norm_kernel<T, ALIGNED, GROUP, BLOCKS, Eight::none>, blocks, kThreads, stream, a);
        case Eight::e4m3: return launch(norm_kernel<T, ALIGNED, GROUP, BLOCKS, Eight::e4m3>, blocks, kThreads, stream, a);
        default: return launch(norm_kernel<T, ALIGNED, GROUP, BLOCKS, Eight::int8>, blocks, kThreads, stream, a);
    }
}

// A wave a row while a lane needs at most four vectors (no barrier, four rows a workgroup), then a
// workgroup of 256, then one of 1024 lanes, then the form that reads the row again.
// A group of lanes as wide as its row, with four vectors a lane: a wider one idles and has to meet at
// barriers. 20 million bfloat16 elements with a residual in groups of 64, 256 and 1024 lanes: rows of 256
// 32, 82 and 293 us, of 1024 27, 31 and 78, of 2048 27, 26 and 43, of 8192 (256 and 1024) 26.6 and 26.5.
// Rows of 32768 take 27.2 us out of registers and 36.1 read again; to e4m3, read three times, 29.9 and 45.6.
template <typename T, bool ALIGNED>
hipError_t by_width(const NormArgs &a, Eight eight, hipStream_t stream) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int vectors = (a.width + V - 1) / V;
    if (vectors <= 4 * 64) return run<T, ALIGNED, 64, 4>(a, eight, stream);
    if (vectors <= 4 * 256) return run<T, ALIGNED, 256, 4>(a, eight, stream);
    if (vectors <= 4 * 1024) return run<T, ALIGNED, 1024, 4>(a, eight, stream);
    return run<T, ALIGNED, 1024, 0>(a, eight, stream);
}

template <typename T>
hipError_t by_alignment(const NormArgs &a, Eight eight, hipStream_t stream) {
    constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                           reinterpret_cast<uintptr_t>(a.weight) | reinterpret_cast<uintptr_t>(a.residual_out) |
                           reinterpret_cast<uintptr_t>(a.y);
    const size_t strides = a.x_stride | a.residual_stride | a.residual_out_stride | a.y_stride | a.q_stride;
    // vectors at any element cost rows of 256 33 us in place of 31.5, of 2048 27.7 for 26.9, of 32768 31.2 for 27.2
    const bool wide = bits % 16 == 0 && reinterpret_cast<uintptr_t>(a.q) % kVec == 0 && a.width % kVec == 0 &&
                      strides % kVec == 0;
    return wide ? by_width<T, true>(a, eight, stream) : by_width<T, false>(a, eight, stream);
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs &a, Elem type, Eight eight, hipStream_t stream) {
    if (a.rows <= 0) return hipSuccess;
    switch (type) {
        case Elem::f32: return by_alignment<float>(a, eight, stream);
        case Elem::bf16: return by_alignment<__bf16>(a, eight, stream);
        default: return by_alignment<_Float16>(a, eight, stream);
    }
}

}  // namespace bl
