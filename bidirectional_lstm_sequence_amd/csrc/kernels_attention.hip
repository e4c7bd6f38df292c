// Cross attention: rows of packed sequences, or one row a sequence, read memories of frames.
//
//   s[f] = scale q . k[f];  y = sum_f e^(s[f] - m) v[f] / sum_f e^(s[f] - m),  m about max_f s[f]
//
// in one pass over the frames with a running reference m and sum. The heads that share keys and values are packed rows
// of one tile. Both products run on 32 x 32 matrix instructions with frames as rows of the first result, so that a lane
// holds weights of its own row alone and hands them to the second product as they lie; values are read from LDS by
// columns. Tiles of keys and values go straight from memory to two stages of LDS; frames that do not count come as zeros
// (an offset behind the buffer) and their scores become minus infinity, so neither what they hold nor what a query makes of
// the zeros enters.
//
// Few rows are bound by the bytes of keys and values: 256 rows over 589 frames each, 4 key heads of 64, bfloat16, 35
// us (floor 31 at the copy rate of 5.0 TB/s); 64 rows over 4096 frames, 8 key heads of 128, 186 us, 5.8 TB/s. Many rows:
// 16384 over 2048 frames, 32 heads of 128, bfloat16, 803 us, 685 TFLOP/s, half as many matrix operations again for the
// weights' second part (610 us without). Matrix instructions alone, with neither loads nor softmax, take 482; of the rest, in
// trials that leave one out, reads from LDS 217 us, loads to LDS 80, softmax 62.
// float32 takes the float32 matrix instructions: 4096 rows, 8 heads of 128, 287 us, 120 TFLOP/s of 138.
#include "attention_device.h"

namespace bl {
namespace {

// A workgroup has either 128 or 256 packed rows, 32 a wave, and its waves read tiles of frames together (many); or up
// to 32 packed rows, and its waves read every fourth tile each, whose sums they join (few). Many with keys of RB = 512
// bytes take eight waves, so that two share a SIMD: 575 us where four take 667 (8192 rows, 16 heads of 256).
template <bool FEW, int RB>  // few: as many as have two tiles of 32 frames in 128 KB
constexpr int kWaves = FEW ? (RB <= 256 ? 4 : (RB == 512 ? 2 : 1)) : (RB == 512 ? 8 : 4);

template <bool FEW, int RB>
constexpr int kRows = FEW ? 32 : 32 * kWaves<FEW, RB>;

// Rows of RB bytes in LDS: chunk c of 16 bytes of row r lies at place(r, c), so that what one instruction reads falls
// on all 64 banks. Keys are read a chunk of 32 rows at a time; values four rows by 64 bytes, or in float32 two rows,
// four apart, by 128.
template <int RB>
__device__ __forceinline__ int key_place(int r, int c) {
    return RB >= 256 ? c ^ (r & 15) : (RB == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3));
}

template <typename T, int RB>
__device__ __forceinline__ int value_place(int r, int c) {
    if constexpr (sizeof(T) == 4) return RB >= 256 ? c ^ (r & 4) << 1 : c;
    return RB >= 256 ? c ^ (r & 3) << 2 : (RB == 128 ? c ^ (r & 2) << 1 : c);
}

// The same places from a lane's first one: chunk c of a row whose chunk `half` is at `at`, for even c - half, and a lane's
// values 32 d columns further than `at`. What places exchange is a few bits of the chunk, so one exclusive or of a constant
// finds them. (A register for every place made heads of 256 bfloat16 spill in the loop, 1.5 times as long.)
template <int RB>
__device__ __forceinline__ int key_at(int at, int c) {
    constexpr int kTurns = RB >= 256 ? 15 : (RB == 128 ? 7 : 3);
    return (at ^ (c & kTurns) * 16) + (c & ~kTurns) * 16;
}

template <typename T, int RB>
__device__ __forceinline__ int values_at(int at, int d) {
    constexpr int kTurns = sizeof(T) == 4 ? (RB >= 256 ? 1 : 0) : (RB >= 256 ? 3 : (RB == 128 ? 1 : 0));
    constexpr int kBytes = 32 * static_cast<int>(sizeof(T));
    return (at ^ (d & kTurns) * kBytes) + (d & ~kTurns) * kBytes;
}

// Products of 32 x 32. A fragment of keys or queries: row lane % 32, chunk 2 s + lane / 32 of 16 bytes.
// The first product gives frames by rows: a lane holds of its row, lane % 32, the frames
// 8 (i / 4) + 4 (lane / 32) + i % 4 in i = 0 .. 15. That is how the second product takes them, with the values'
// frames in the same order, so that weights never leave their lane.
template <typename T>
struct Of {
    typedef Vec<T, 8> Frag;
    static constexpr int kFrames = 64;  // of a tile
    // Weights are e^(s - m) times 2^kLift, for an m within 2^kLag of the largest: those of fp16 keep their 11 bits
    // down to 2^-24 of the largest and stay below 2^15.
    static constexpr float kLift = __is_same(T, _Float16) ? 10.0f : 0.0f;
    static constexpr float kLag = __is_same(T, _Float16) ? 5.0f : 8.0f;
    static __device__ __forceinline__ F16x mul(const Frag &a, const Frag &b, const F16x &c) {
        if constexpr (__is_same(T, __bf16)) {
            return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
        } else {
            return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
        }
    }
    // Four rows by columns: 16 lanes name four elements each of rows r .. r + 3 and receive a column. Lane's place for the
    // first 32 columns of the rows 4 (lane / 32) on; 32 columns further it is `values_at`'s.
    template <int RB>
    static __device__ __forceinline__ int values_from(int lane) {
        const int row = 4 * (lane >> 5) + ((lane & 15) >> 2), c = 16 * (lane >> 4 & 1) + 4 * (lane & 3);
        return row * RB + value_place<T, RB>(row, c >> 3) * 16 + (c & 7) * 2;
    }
    static __device__ __forceinline__ Vec<T, 4> columns(const char *p) {
        typedef short S4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) S4 *Lds;
        return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
    }
    // 32 frames' weights as the second product takes them, in two parts: rounded, and what the rounding left (2^-16 of a
    // weight is lost then, no more than float32's 24 bits need for an output of 16). Their sum is that of both parts. A
    // bfloat16 row over 589 frames is off by 0.0017 of its size so, which is the output's own rounding, by 0.0023 with one
    // part; values that nearly cancel show the difference at any size.
    struct Weights {
        Frag part[2][2];
    };
    static __device__ __forceinline__ Weights pack(const F16x &p, float &sum) {
        Weights w;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float a = p[8 * c + j], b = p[8 * c + j + 1];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const Vec<T, 2> pair = {static_cast<T>(a), static_cast<T>(b)};
                    const Vec<T, 2> ones = {static_cast<T>(1.0f), static_cast<T>(1.0f)};
                    if constexpr (__is_same(T, __bf16)) {
                        sum = __builtin_amdgcn_fdot2_f32_bf16(pair, ones, sum, false);
                    } else {
                        sum = __builtin_amdgcn_fdot2(pair, ones, sum, false);
                    }
                    w.part[k][c][j] = pair[0];
                    w.part[k][c][j + 1] = pair[1];
                    a -= static_cast<float>(pair[0]);
                    b -= static_cast<float>(pair[1]);
                }
            }
        return w;
    }
    // Infinities as zeros, for the second part of weights: it may be zero or below, what the first part gives is right.
    static __device__ __forceinline__ Frag finite(const Frag &v) {
        typedef unsigned short U8 __attribute__((ext_vector_type(8)));
        constexpr unsigned short kInfinity = __is_same(T, __bf16) ? 0x7F80 : 0x7C00;
        U8 bits = __builtin_bit_cast(U8, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) bits[e] = (bits[e] & 0x7FFF) == kInfinity ? 0 : bits[e];
        return __builtin_bit_cast(Frag, bits);
    }
    // out[d] += values' columns 32 d .. 32 d + 31 of 32 frames from r on, times their weights; `at`: values_from's place
    template <int RB, bool AGAIN, int N>
    static __device__ __forceinline__ void weigh(const char *values, int at, int r, const Weights &w, F16x (&out)[N]) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int d = 0; d < N; ++d) {
                const char *const p = values + values_at<T, RB>(at, d) + (r + 16 * c) * RB;
                const Frag v = __builtin_shufflevector(columns(p), columns(p + 8 * RB), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int k = 0; k < 2; ++k) out[d] = mul(AGAIN && k > 0 ? finite(v) : v, w.part[k][c], out[d]);
            }
    }
};

template <>
struct Of<float> {
    typedef Vec<float, 4> Frag;
    static constexpr int kFrames = 32;
    static constexpr float kLift = 0.0f, kLag = 8.0f;
    using Weights = F16x;
    static __device__ __forceinline__ F16x pack(const F16x &p, float &sum) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += p[i];
        return p;
    }
    static __device__ __forceinline__ F16x mul(const Frag &a, const Frag &b, F16x c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    template <int RB>
    static __device__ __forceinline__ int values_from(int lane) {
        const int row = 4 * (lane >> 5), c = lane & 31;
        return row * RB + value_place<float, RB>(row, c >> 2) * 16 + (c & 3) * 4;
    }
    template <int RB, bool, int N>
    static __device__ __forceinline__ void weigh(const char *values, int at, int r, const F16x &p, F16x (&out)[N]) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int d = 0; d < N; ++d) {
                const float v = __uint_as_float(
                    *reinterpret_cast<const unsigned *>(values + values_at<float, RB>(at, d) + (r + 8 * (i / 4) + i % 4) * RB));
                out[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, p[i], out[d], 0, 0, 0);
            }
    }
};

__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }

// e^(scale d) times 2^lift for a difference d of two products' sums: scores of any size, whose product with log2 e need not
// be a float32, give the exponents that their difference does. float32 tensors carry the rest of the factor and of its
// product along (as exp_of_minus does), so that the exponent is that of a rounded difference alone.
struct Power {
    float high, low;
    __device__ __forceinline__ explicit Power(float scale) {
        constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.9259629911266175e-8f;
        high = scale * kLog2e;
        low = fmaf(scale, kLog2e, -high) + scale * kLog2eLow;
    }
    template <typename T>
    __device__ __forceinline__ float of(float d, float lift = 0.0f) const {
        if constexpr (sizeof(T) == 4) {
            const float t = d * high, e = __builtin_amdgcn_exp2f(t);
            const float rest = fmaf(d, high, -t) + d * low;
            return e > 0.0f ? fmaf(e, rest * 0.6931471805599453f, e) : e;
        } else {
            return __builtin_amdgcn_exp2f(fmaf(d, high, lift));
        }
    }
};

struct First {
    static constexpr bool value = false;
};
struct Again {
    static constexpr bool value = true;
};

// D: columns of a tile, the width rounded up; columns behind the width are zeros.
template <typename T, int D, bool FEW, bool ALIGNED>
__global__ __launch_bounds__((64 * kWaves<FEW, D * sizeof(T)>), (!FEW && D * sizeof(T) <= 512 ? 2 : 1)) void attention_kernel(AttentionArgs a) {
    typedef Of<T> O;
    constexpr int kSize = static_cast<int>(sizeof(T)), kPer = 16 / kSize;
    constexpr int RB = D * kSize;
    constexpr int kFrames = FEW || D == 256 ? 32 : O::kFrames;
    constexpr int kTile = kFrames * RB;  // bytes of a tile's keys, and of its values
    constexpr int kAll = kWaves<FEW, RB>, kSharers = FEW ? 1 : kAll;  // waves; those that bring a tile
    constexpr int kLoads = kTile / 1024 / kSharers;
    constexpr int kSlabs = RB / 32;
    constexpr int kBlocks = kFrames / 32, kColumns = D / 32;
    static_assert(kTile % (1024 * kSharers) == 0, "whole instructions a wave");
    __shared__ __attribute__((aligned(1024))) char lds_of_all[2 * 2 * kTile * (FEW ? kAll : 1)];

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sharer = FEW ? 0 : wave;
    char *const lds = lds_of_all + (FEW ? wave * 4 * kTile : 0);
    const Work w = work_of(a, kRows<FEW, RB>, kFrames);
    if (w.count == 0) return;  // uniform

    // this lane's row, and its queries
    const int at = sharer * 32 + (lane & 31);
    const bool real = at < w.count;
    const long long packed = w.first + (real ? at : 0);
    const long long row = w.row + packed / a.per;
    const int head = w.group * a.per + static_cast<int>(packed % a.per);
    const T *const q = static_cast<const T *>(a.q) + static_cast<size_t>(row) * a.q_stride + static_cast<size_t>(head) * a.width;
    typename O::Frag qf[kSlabs];
#pragma unroll
    for (int s = 0; s < kSlabs; ++s) {
        const int c = (2 * s + half) * kPer;
        qf[s] = __builtin_bit_cast(typename O::Frag, load_vector<false, T, kPer>(q + c, a.width - c));
    }

    const T *const k = static_cast<const T *>(a.k) + static_cast<size_t>(w.memory) * a.k_stride + static_cast<size_t>(w.group) * a.width;
    const T *const v = static_cast<const T *>(a.v) + static_cast<size_t>(w.memory) * a.v_stride + static_cast<size_t>(w.group) * a.width;
    const unsigned char *const mask = a.mask != nullptr ? a.mask + w.memory : nullptr;

    // Which of 64 frames from f on count: bit i is frame f + i. `byte` is the mask's for frame f + lane.
    auto mask_byte = [&](int f) -> int { return mask != nullptr && f + lane < w.end ? mask[f + lane] : 1; };
    auto counted = [&](int f, int byte) -> unsigned long long {
        return __ballot(f + lane < w.end && lane < kFrames && byte != 0);
    };

    constexpr unsigned long long kWhole = kFrames == 64 ? ~0ull : (1ull << kFrames) - 1;
    int load_row[kLoads], key_chunk[kLoads], value_chunk[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int byte = (i * kSharers + sharer) * 1024 + lane * 16;
        load_row[i] = byte / RB;
        key_chunk[i] = key_place<RB>(load_row[i], byte % RB / 16);
        value_chunk[i] = value_place<T, RB>(load_row[i], byte % RB / 16);
    }
    unsigned key_offset[ALIGNED ? kLoads : 1], value_offset[ALIGNED ? kLoads : 1];
    if constexpr (ALIGNED) {
        const int bytes = a.width * kSize;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int kc = 16 * key_chunk[i], vc = 16 * value_chunk[i];
            key_offset[i] = kc < bytes ? static_cast<unsigned>(load_row[i] * a.k_stride * kSize) + kc : kOutOfRange;
            value_offset[i] = vc < bytes ? static_cast<unsigned>(load_row[i] * a.v_stride * kSize) + vc : kOutOfRange;
        }
    }
    auto issue = [&](int slot, int f, unsigned long long bits) __attribute__((always_inline)) {
        if constexpr (ALIGNED) {
            const T *const kt = k + static_cast<size_t>(f) * a.k_stride, *const vt = v + static_cast<size_t>(f) * a.v_stride;
            char *const base = lds + slot * 2 * kTile + sharer * 1024;
            if (bits == kWhole) {  // uniform
#pragma unroll
                for (int i = 0; i < kLoads; ++i) load_to_lds(kt, base + i * kSharers * 1024, key_offset[i], 0);
#pragma unroll
                for (int i = 0; i < kLoads; ++i) load_to_lds(vt, base + kTile + i * kSharers * 1024, value_offset[i], 0);
            } else {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const bool in = bits >> load_row[i] & 1;
                    load_to_lds(kt, base + i * kSharers * 1024, in ? key_offset[i] : kOutOfRange, 0);
                    load_to_lds(vt, base + kTile + i * kSharers * 1024, in ? value_offset[i] : kOutOfRange, 0);
                }
            }
        }
    };
    U4 held_keys[ALIGNED ? 1 : kLoads], held_values[ALIGNED ? 1 : kLoads];
    auto fetch = [&](int f, unsigned long long bits) __attribute__((always_inline)) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const bool in = bits >> load_row[i] & 1;
                const int kc = key_chunk[i] * kPer, vc = value_chunk[i] * kPer;
                const size_t r = static_cast<size_t>(f) + load_row[i];
                held_keys[i] = __builtin_bit_cast(U4, load_vector<false, T, kPer>(k + r * a.k_stride + kc, in ? a.width - kc : 0));
                held_values[i] = __builtin_bit_cast(U4, load_vector<false, T, kPer>(v + r * a.v_stride + vc, in ? a.width - vc : 0));
            }
        }
    };
    auto put = [&](int slot) __attribute__((always_inline)) {
        if constexpr (!ALIGNED) {
            char *const base = lds + slot * 2 * kTile + sharer * 1024 + lane * 16;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                *reinterpret_cast<U4 *>(base + i * kSharers * 1024) = held_keys[i];
                *reinterpret_cast<U4 *>(base + kTile + i * kSharers * 1024) = held_values[i];
            }
        }
    };

    // Weights up to 2^kLag times values near the end of float32 leave it, and an infinite value times the second part of a
    // weight is no number: where a sum is not finite, its workgroup (of few rows: its wave) goes over the frames a second
    // time, AGAIN, with weights times `lower`, so that no sum of the values' type leaves float32 (fp16's never do), and
    // infinities out of the second part. Sums that were finite come out the same, times `lower`.
    const Power power(a.scale);
    const int room = __is_same(T, _Float16) || w.end <= w.begin ? 0 : static_cast<int>(O::kLag) + 33 - __builtin_clz(w.end - w.begin);
    const float lower = __builtin_ldexpf(1.0f, -room);
    float most, sum;  // sum: this half's frames
    F16x out[kColumns];

    const int key_from = (lane & 31) * RB + key_place<RB>(lane & 31, half) * 16, value_from = O::template values_from<RB>(lane);
    auto tile = [&](auto again, int slot, unsigned long long bits) __attribute__((always_inline)) {
        constexpr bool AGAIN = decltype(again)::value;
        const int keys = slot * 2 * kTile + key_from, values = slot * 2 * kTile + kTile + value_from;
        __builtin_amdgcn_s_setprio(1);
        F16x p[kBlocks];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) p[b] = F16x{};
#pragma unroll
        for (int i = 0; i < kSlabs; ++i)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                // read as integers: before floats from LDS the compiler waits for all loads to LDS under way
                const U4 chunk = *reinterpret_cast<const U4 *>(lds + key_at<RB>(keys, 2 * i) + b * 32 * RB);
                p[b] = O::mul(__builtin_bit_cast(typename O::Frag, chunk), qf[i], p[b]);
            }
        __builtin_amdgcn_s_setprio(0);
        if (bits != kWhole) {  // uniform; what came of the zeros of keys that do not count is no number where a query is not
            const unsigned long long mine = bits >> 4 * half;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) p[b][i] = mine >> (32 * b + 8 * (i / 4) + i % 4) & 1 ? p[b][i] : -__builtin_huge_valf();
        }
        float top = -__builtin_huge_valf();
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, p[b][i]);
        top = fmaxf(top, other_half(top));
        // Weights are measured from `most`, which follows a row's maximum only where that is kLag further up: its sums and
        // values then move with it. They rarely have to, and a wave whose rows stay skips it.
        const bool moves = (top - most) * power.high > O::kLag;  // also from minus infinity; never where both are
        if (__any(moves)) {
            const float next = moves ? top : most;
            const float down = !moves ? 1.0f : (most == -__builtin_huge_valf() ? 0.0f : power.of<T>(most - next));
            most = next;
            sum *= down;
#pragma unroll
            for (int d = 0; d < kColumns; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) out[d][i] *= down;
        }
        const float from = most == -__builtin_huge_valf() ? 0.0f : most;  // no frame yet: weights of 0
        float add = 0.0f;
        typename O::Weights weights[kBlocks];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[b][i] = power.of<T>(p[b][i] - from, O::kLift);
                if constexpr (AGAIN) p[b][i] *= lower;
            }
            weights[b] = O::pack(p[b], add);
        }
        sum += add;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) O::template weigh<RB, AGAIN>(lds, values, 32 * b, weights[b], out);
    };

    constexpr int kStride = FEW ? kAll * kFrames : kFrames;
    const int begin = w.begin + (FEW ? wave * kFrames : 0);
    auto pass = [&](auto again) __attribute__((always_inline)) {
        most = -__builtin_huge_valf(), sum = 0.0f;
#pragma unroll
        for (int d = 0; d < kColumns; ++d) out[d] = F16x{};
        if (begin < w.end) {  // uniform where waves meet
            unsigned long long bits = counted(begin, mask_byte(begin));
            int next_byte = mask_byte(begin + kStride);
            if constexpr (ALIGNED) {
                issue(0, begin, bits);
            } else {
                fetch(begin, bits);
            }
            for (int f = begin, slot = 0; f < w.end; f += kStride, slot ^= 1) {
                const bool more = w.end - f > kStride;
                const unsigned long long next = more ? counted(f + kStride, next_byte) : 0;
                if constexpr (ALIGNED) {
                    meet<0, !FEW>();  // the tile has landed, and every wave is done with the other one
                    if (more) issue(slot ^ 1, f + kStride, next);
                } else {
                    put(slot);
                    if constexpr (FEW) {
                        own_lds();
                    } else {
                        __syncthreads();
                    }
                    if (more) fetch(f + kStride, next);
                }
                if (w.end - f > 2 * kStride) next_byte = mask_byte(f + 2 * kStride);
                tile(again, slot, bits);
                bits = next;
            }
        }
        sum += other_half(sum);
    };
    pass(First{});
    bool odd = !(sum < __builtin_huge_valf());
#pragma unroll
    for (int d = 0; d < kColumns; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) odd |= !(fabsf(out[d][i]) < __builtin_huge_valf());
    float back = 1.0f;
    bool again = __any(odd);
    if constexpr (!FEW) {  // by floats in LDS: with __syncthreads_or the compiler lets each tile's reads wait for the next one's loads
        float *const odds = reinterpret_cast<float *>(lds_of_all);
        meet<0>();  // every wave is done with the tiles
        if (lane == 0) odds[wave] = again ? 1.0f : 0.0f;
        meet<0>();
        float any = 0.0f;
#pragma unroll
        for (int u = 0; u < kAll; ++u) any += odds[u];
        again = any > 0.0f;
    }
    if (again) {
        if constexpr (!FEW) meet<0>();
        pass(Again{});
        back = __builtin_ldexpf(1.0f, room);
    }

    // from here on `out` is the quotient: parts are joined by their shares, and no share passes a value
    const float inverse = 1.0f / sum;
#pragma unroll
    for (int d = 0; d < kColumns; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) out[d][i] = sum == 0.0f ? 0.0f : out[d][i] * inverse;  // no frame: zeros
    sum *= back;
    if constexpr (FEW) {
        // every wave's share of the rows to its own LDS, and from there to whole lines
        constexpr int kRow = D + 4;  // floats: the padding spreads rows over the banks
        constexpr int kShare = kTile;  // floats from one wave's share to the next
        static_assert((32 * kRow + 64) * 4 <= 4 * kTile, "a share fits the wave's tiles");
        float *const mine = reinterpret_cast<float *>(lds), *const shares = reinterpret_cast<float *>(lds_of_all);
        own_lds();
#pragma unroll
        for (int d = 0; d < kColumns; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                *reinterpret_cast<Vec<float, 4> *>(mine + at * kRow + 32 * d + 2 * i + 4 * half) = {out[d][i], out[d][i + 1], out[d][i + 2],
                                                                                                    out[d][i + 3]};
            }
        if (half == 0) *reinterpret_cast<Vec<float, 2> *>(mine + 32 * kRow + 2 * at) = {most, sum};
        __syncthreads();
        for (int item = threadIdx.x; item < w.count * (D / 4); item += 64 * kAll) {
            const int r = item / (D / 4), col = item % (D / 4) * 4;
            if (col >= a.width) continue;
            float top = -__builtin_huge_valf(), total = 0.0f, part[kAll];
#pragma unroll
            for (int u = 0; u < kAll; ++u) top = fmaxf(top, shares[u * kShare + 32 * kRow + 2 * r]);
            const float from = top == -__builtin_huge_valf() ? 0.0f : top;
#pragma unroll
            for (int u = 0; u < kAll; ++u) {
                const float *const mine_of = shares + u * kShare + 32 * kRow + 2 * r;
                part[u] = mine_of[1] * power.of<T>(mine_of[0] - from);
                total += part[u];
            }
            const float inverse_total = total == 0.0f ? 0.0f : 1.0f / total;
            Vec<float, 4> value = {};
#pragma unroll
            for (int u = 0; u < kAll; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) value[e] = fmaf(shares[u * kShare + r * kRow + col + e], part[u] * inverse_total, value[e]);
            const long long packed_r = w.first + r, row_r = w.row + packed_r / a.per;
            const int head_r = w.group * a.per + static_cast<int>(packed_r % a.per);
            if (a.splits > 1) {
                *reinterpret_cast<Vec<float, 4> *>(part_values(a, w.split, row_r, head_r) + col) = value;
                if (col == 0) *reinterpret_cast<Vec<float, 2> *>(part_sums(a, w.split, row_r, head_r)) = {top, total};
            } else {
                Vec<T, 4> four;
#pragma unroll
                for (int e = 0; e < 4; ++e) four[e] = static_cast<T>(value[e]);
                T *const y = static_cast<T *>(a.y) + static_cast<size_t>(row_r) * a.y_stride + static_cast<size_t>(head_r) * a.width;
                store_vector<false, T, 4>(y + col, four, a.width - col);
            }
        }
        return;
    }
    if (!real) return;
    if (a.splits > 1) {
        float *const part = part_values(a, w.split, row, head);
#pragma unroll
        for (int d = 0; d < kColumns; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int col = 32 * d + 2 * i + 4 * half;
                if (col < a.padded) *reinterpret_cast<Vec<float, 4> *>(part + col) = {out[d][i], out[d][i + 1], out[d][i + 2], out[d][i + 3]};
            }
        if (half == 0) *reinterpret_cast<Vec<float, 2> *>(part_sums(a, w.split, row, head)) = {most, sum};
        return;
    }
    T *const y = static_cast<T *>(a.y) + static_cast<size_t>(row) * a.y_stride + static_cast<size_t>(head) * a.width;
#pragma unroll
    for (int d = 0; d < kColumns; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int col = 32 * d + 2 * i + 4 * half;
            Vec<T, 4> four;
#pragma unroll
            for (int e = 0; e < 4; ++e) four[e] = static_cast<T>(out[d][i + e]);
            if (col < a.width) store_vector<false, T, 4>(y + col, four, a.width - col);
        }
}

// The parts of up to kJoinRows packed rows of one group, by their shares of all weights. Four columns a lane.
constexpr int kJoinRows = 16;

template <typename T>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a) {
    const int splits = a.splits;
    const Power power(a.scale);
    AttentionArgs whole = a;
    whole.splits = 1;
    const Work w = work_of(whole, kJoinRows, 1);
    const int lanes = a.padded / 4;
    for (int item = threadIdx.x; item < w.count * lanes; item += 256) {
        const long long packed = w.first + item / lanes;
        const int col = item % lanes * 4;
        const long long row = w.row + packed / a.per;
        const int head = w.group * a.per + static_cast<int>(packed % a.per);
        float top = -__builtin_huge_valf();
#pragma unroll 4
        for (int s = 0; s < splits; ++s) top = fmaxf(top, part_sums(a, s, row, head)[0]);
        const float from = top == -__builtin_huge_valf() ? 0.0f : top;
        auto share = [&](int s) {
            const Vec<float, 2> part = *reinterpret_cast<const Vec<float, 2> *>(part_sums(a, s, row, head));
            return part[1] * power.of<T>(part[0] - from);
        };
        float total = 0.0f;
#pragma unroll 4
        for (int s = 0; s < splits; ++s) total += share(s);
        const float inverse = total == 0.0f ? 0.0f : 1.0f / total;
        Vec<float, 4> v = {};
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const Vec<float, 4> add = *reinterpret_cast<const Vec<float, 4> *>(part_values(a, s, row, head) + col);
            const float weight = share(s) * inverse;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(add[e], weight, v[e]);
        }
        T *const y = static_cast<T *>(a.y) + static_cast<size_t>(row) * a.y_stride + static_cast<size_t>(head) * a.width;
        Vec<T, 4> four;
#pragma unroll
        for (int e = 0; e < 4; ++e) four[e] = static_cast<T>(v[e]);
        store_vector<false, T, 4>(y + col, four, a.width - col);
    }
}

unsigned long long tiles_of(const AttentionArgs &a, int size) {
    if (a.step) return static_cast<unsigned long long>(a.seq.sequences) * ((a.per + size - 1) / size);
    return static_cast<unsigned long long>(a.seq.rows) * a.per / size + a.seq.sequences;
}

// Whether a sequence has 32 packed rows or less on average: 256 rows of 16 heads on 4 over 589 frames take 35 us so and 49
// with tiles of 128, a row alone 11 and 15. With 64 packed rows the tiles of 128 are ahead (8 x 64 rows over 2048 frames,
// heads of 128, 31.6 us and 33.5; 32 x 64 rows of float32 over 589 frames 36.5 and 40.8). The lengths are on the device: a
// long sequence among many short ones is read by workgroups of 32: a prompt of 4000 rows adds 130 us to 255 single rows'
// 382, alone it takes 73.
bool few_rows(const AttentionArgs &a) {
    return static_cast<unsigned long long>(a.seq.rows) * a.per <= 32ull * a.seq.sequences;
}

// Frames are split over workgroups where those are few, by what the average sequence and memory have, up to two
// workgroups a CU: one prompt of 500 rows over 4096 frames 30 us with 8 splits, 36 with 16 and their larger join; 32 x 4
// rows over 4096 frames 111 us with 2, 141 with none. A split keeps at least four tiles for each wave of the few, and
// two of the many.
int splits_of(const AttentionArgs &a) {
    const bool few = few_rows(a);
    const unsigned long long each = (static_cast<unsigned long long>(a.seq.rows) * a.per + a.seq.sequences - 1) / a.seq.sequences;
    const unsigned long long size = few ? 32 : 128, work = (each + size - 1) / size * a.seq.sequences * a.groups;
    const long long frames = a.seq.places > 0 ? a.memory_rows / a.seq.places : 0, least = few ? 512 : 128;
    int splits = 1;
    while (splits < 16 && work * splits * 2 <= 512 && frames / (splits * 2) >= least) splits *= 2;
    return splits;
}

template <typename T, int D, bool FEW, bool ALIGNED>
hipError_t run(AttentionArgs a, hipStream_t stream) {
    a.splits = splits_of(a);
    a.padded = (a.width + 3) / 4 * 4;
    const hipError_t e = launch(attention_kernel<T, D, FEW, ALIGNED>, tiles_of(a, kRows<FEW, D * sizeof(T)>) * a.groups * a.splits,
                                64 * kWaves<FEW, D * sizeof(T)>, stream, a);
    if (e != hipSuccess || a.splits == 1) return e;
    return launch(attention_join_kernel<T>, tiles_of(a, kJoinRows) * a.groups, 256, stream, a);
}

template <typename T, bool FEW, bool ALIGNED>
hipError_t by_width(const AttentionArgs &a, hipStream_t stream) {
    if (a.width <= 32) return run<T, 32, FEW, ALIGNED>(a, stream);
    if (a.width <= 64) return run<T, 64, FEW, ALIGNED>(a, stream);
    if (a.width <= 128) return run<T, 128, FEW, ALIGNED>(a, stream);
    return run<T, 256, FEW, ALIGNED>(a, stream);
}

template <typename T, bool ALIGNED>
hipError_t by_rows(const AttentionArgs &a, hipStream_t stream) {
    return few_rows(a) ? by_width<T, true, ALIGNED>(a, stream) : by_width<T, false, ALIGNED>(a, stream);
}

template <typename T>
hipError_t by_alignment(const AttentionArgs &a, hipStream_t stream) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          (a.k_stride | a.v_stride | static_cast<uint64_t>(a.width)) * sizeof(T);
    const uint64_t longest = (a.k_stride > a.v_stride ? a.k_stride : a.v_stride) * sizeof(T);
    return bits % 16 == 0 && longest <= kBufferBytes / 128 ? by_rows<T, true>(a, stream) : by_rows<T, false>(a, stream);
}

}  // namespace

size_t attention_scratch_bytes(const AttentionArgs &a) {
    if (a.seq.rows <= 0 || a.seq.sequences <= 0) return 0;
    const int splits = splits_of(a);
    return splits > 1 ? static_cast<size_t>(splits) * a.seq.rows * a.heads * ((a.width + 3) / 4 * 4 + 2) * 4 : 0;
}

hipError_t launch_attention(const AttentionArgs &a, Elem type, hipStream_t stream) {
    if (a.seq.rows <= 0 || a.seq.sequences <= 0) return hipSuccess;
    switch (type) {
        case Elem::f32: return by_alignment<float>(a, stream);
        case Elem::bf16: return by_alignment<__bf16>(a, stream);
        default: return by_alignment<_Float16>(a, stream);
    }
}

}  // namespace bl
