// Device helpers of the matrix product: operands of its element types, tiles and the epilogue.
#pragma once

#include "tile_device.h"

namespace bl {

typedef float F4 __attribute__((ext_vector_type(4)));
typedef int I4 __attribute__((ext_vector_type(4)));

// A row of a stage holds 128 bytes of its K, chunk c of 16 bytes at place c ^ (row & 7): the rows of a fragment fall
// on all banks.
constexpr int kRowBytes = 128;

// Operands by element type, for products of 16 x 16 (those of 32 x 32 took 2.1 us a step of 256 x 256 x 64 bfloat16,
// these 1.6). A fragment holds, for row lane % 16, what lane / 16 contributes to slab s of K; as both operands number
// K alike, any share of a slab's chunks will do. An accumulator's element e is row 4 (lane / 16) + e of the first
// operand and row lane % 16 of the second. `turned` is row & 7.
template <typename T>
struct Of16 {
    typedef T Elem;
    typedef Vec<T, 8> Frag;
    typedef F4 Acc;
    static constexpr int kSlab = 64;  // bytes of K
    static constexpr bool kScaled = false;
    static constexpr int kChunks = 1;  // of 16 bytes in a fragment
    static __device__ __forceinline__ Frag of(const I4 (&chunk)[1]) { return __builtin_bit_cast(Frag, chunk[0]); }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, const Acc &c) {
        if constexpr (__is_same(T, __bf16)) {
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
        } else {
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
        }
    }
};

struct OfF32 {
    typedef float Elem;
    typedef F4 Frag;
    typedef F4 Acc;
    static constexpr int kSlab = 64;
    static constexpr bool kScaled = false;
    static constexpr int kChunks = 1;  // of 16 bytes in a fragment
    static __device__ __forceinline__ Frag of(const I4 (&chunk)[1]) { return __builtin_bit_cast(Frag, chunk[0]); }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, Acc c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

// float32 by three bf16 parts of each operand, which hold its 24 bits: six products of parts (those left out are below
// 2^-25 of the whole) at sixteen times the rate of float32's. The parts are those of 2^16 times the operand: the last bit of
// the smallest float32, 2^-149, is then 2^-133, bf16's own (the matrix instructions keep subnormal numbers). Sums come 2^32
// times too large. A part of an infinity, or of what bf16 rounds to one, is not a number; a tile with sums that are not
// finite, which those from 2^96 on may be, is computed again by OfF32.
struct OfF32Split {
    static constexpr float kTimes = 0x1p16f, kBack = 0x1p-32f;
    typedef float Elem;
    struct Frag {
        Vec<__bf16, 8> part[3];
    };
    typedef F4 Acc;
    static constexpr int kSlab = 128;
    static constexpr bool kScaled = false;
    static constexpr int kChunks = 2;
    static __device__ __forceinline__ Frag of(const I4 (&chunk)[2]) {
        typedef __bf16 B2 __attribute__((ext_vector_type(2)));
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __int_as_float(chunk[e / 4][e % 4]) * kTimes;
        Frag f;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            I4 bits;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const B2 pair = {static_cast<__bf16>(v[e]), static_cast<__bf16>(v[e + 1])};
                unsigned both = __builtin_bit_cast(unsigned, pair);
                asm("" : "+v"(both));  // opaque, else the compiler rounds a second time to widen
                bits[e / 2] = static_cast<int>(both);
                v[e] -= __uint_as_float(both << 16);
                v[e + 1] -= __uint_as_float(both & 0xFFFF0000u);
            }
            f.part[p] = __builtin_bit_cast(Vec<__bf16, 8>, bits);
        }
        return f;
    }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, Acc c) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[2], b.part[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[0], b.part[2], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[1], b.part[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[1], b.part[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[0], b.part[1], c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[0], b.part[0], c, 0, 0, 0);
    }
};

// e4m3 widened to bf16, exactly, so that products and sums are those of 16 bits. The matrix instructions of 8-bit floats
// have twice the rate, but bring eight neighbouring products to the place of the largest and drop what lies below 2^-13 of
// it (with block scales or without, measured): a small product next to large ones that cancel is lost.
struct OfE4m3 {
    typedef unsigned char Elem;
    struct Frag {
        Vec<__bf16, 8> part[2];
    };
    typedef F4 Acc;
    static constexpr int kSlab = 64;
    static constexpr bool kScaled = true;
    static constexpr int kChunks = 1;
    static __device__ __forceinline__ Frag of(const I4 (&chunk)[1]) {
        Frag f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Vec<__bf16, 2> low = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(chunk[0][e], 1.0f, false);
            const Vec<__bf16, 2> high = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(chunk[0][e], 1.0f, true);
            const int at = e % 2 * 4;
            f.part[e / 2][at] = low[0];
            f.part[e / 2][at + 1] = low[1];
            f.part[e / 2][at + 2] = high[0];
            f.part[e / 2][at + 3] = high[1];
        }
        return f;
    }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, Acc c) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[0], b.part[0], c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[1], b.part[1], c, 0, 0, 0);
    }
};

struct OfInt8 {
    typedef unsigned char Elem;
    typedef I4 Frag;
    typedef I4 Acc;
    static constexpr int kSlab = 64;
    static constexpr bool kScaled = true;
    static constexpr int kChunks = 1;  // of 16 bytes in a fragment
    static __device__ __forceinline__ Frag of(const I4 (&chunk)[1]) { return __builtin_bit_cast(Frag, chunk[0]); }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, const Acc &c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
};

// What lane / 16 contributes to slab s from a stage's row.
template <class P>
__device__ __forceinline__ typename P::Frag staged(const char *row, int s, int quad, int turned) {
    I4 chunk[P::kChunks];
#pragma unroll
    for (int c = 0; c < P::kChunks; ++c) chunk[c] = *reinterpret_cast<const I4 *>(row + ((4 * (s * P::kChunks + c) + quad) ^ turned) * 16);
    return P::of(chunk);
}

// A workgroup's tile: first row and output, and its share first .. end - 1 of the K steps. Number `whole` and those
// behind it are tiles' halves: the lower or upper half of the rows.
struct Tile {
    int m, n, first, end, split;
    bool halved;
};

// Workgroups go to the 8 XCDs in turn. Each XCD takes a range of tiles in a row, eight row tiles by all outputs
// at a time, so that what its L2 holds is used by several of its CUs.
__device__ __forceinline__ Tile tile_of(const LinearArgs &a, int bm, int bn) {
    const unsigned total = static_cast<unsigned>(a.tiles_m) * a.tiles_n;
    unsigned number = workgroup_number();
    Tile tile;
    const unsigned whole = static_cast<unsigned>(a.whole);
    const unsigned split = a.splits > 1 ? number / total : 0;
    tile.split = static_cast<int>(split);
    tile.halved = number >= whole;
    tile.first = static_cast<int>(static_cast<long long>(a.steps) * split / a.splits);
    tile.end = static_cast<int>(static_cast<long long>(a.steps) * (split + 1) / a.splits);
    unsigned lower = 0;
    number -= split * total;
    if (tile.halved) {
        lower = (number - whole) & 1;
        number = whole + (number - whole) / 2;
    }
    if (split >= static_cast<unsigned>(a.splits) || number >= total) {
        tile.m = a.rows;  // a number behind the last one
        tile.n = tile.first = tile.end = 0;
        return tile;
    }
    const unsigned per = total / 8, rest = total % 8, xcd = number % 8, at = number / 8;
    const unsigned t = xcd * per + (xcd < rest ? xcd : rest) + at;
    constexpr unsigned kGroup = 8;
    const unsigned wide = kGroup * a.tiles_n, group = t / wide, inside = t - group * wide;
    const unsigned left = a.tiles_m - group * kGroup, high = left < kGroup ? left : kGroup;
    tile.m = static_cast<int>(group * kGroup + inside % high) * bm + static_cast<int>(lower) * bm / 2;
    tile.n = static_cast<int>(inside / high) * bn;
    return tile;
}

__device__ __forceinline__ float *part_of(const LinearArgs &a, int split, int row, int out) {
    const size_t width = (static_cast<size_t>(a.out) + 3) / 4 * 4;
    return a.scratch + (static_cast<size_t>(split) * a.rows + row) * width + out;
}

// v times the normal distribution's integral, by e^(z^2) erfc(z) = t P(t), t = 1 / (1 + c z), z = |v| / sqrt 2. P is
// a fit of the least relative error for z of 0 .. 14, where e^(-z^2) vanishes: 2.5e-8 (degree 8) for float32,
// 1.0e-6 (degree 6), 2^-19, for 16 bits. Nothing cancels: the tail of negative v keeps its digits.
template <typename Y>
__device__ __forceinline__ float gelu(float v) {
    const float u = fabsf(v);
    float t, p;
    if constexpr (sizeof(Y) == 4) {
        t = __builtin_amdgcn_rcpf(fmaf(u, 0.38f * 0.70710678f, 1.0f));
        p = fmaf(0.0584217790f, t, -0.2598602861f);
        p = fmaf(p, t, 0.3593385990f);
        p = fmaf(p, t, -0.1568387683f);
        p = fmaf(p, t, 0.2272185822f);
        p = fmaf(p, t, 0.1396805625f);
        p = fmaf(p, t, 0.2036852319f);
        p = fmaf(p, t, 0.2139444557f);
        p = fmaf(p, t, 0.2144098326f);
    } else {
        t = __builtin_amdgcn_rcpf(fmaf(u, 0.38f * 0.70710678f, 1.0f));
        p = fmaf(-0.1254189850f, t, 0.3360414801f);
        p = fmaf(p, t, -0.0699207990f);
        p = fmaf(p, t, 0.2478400746f);
        p = fmaf(p, t, 0.1805920497f);
        p = fmaf(p, t, 0.2165778670f);
        p = fmaf(p, t, 0.2142872767f);
    }
    const float tail = 0.5f * (p * t) * __builtin_amdgcn_exp2f(-0.72134752f * (v * v));
    const float part = v < 0.0f ? tail : 1.0f - tail;
    return v == -__builtin_huge_valf() ? 0.0f : v * part;
}

template <typename Y>
__device__ __forceinline__ float activate(float v, int kind, float slope) {
    switch (kind) {
        case 1: return __builtin_elementwise_maximum(v, 0.0f);
        case 2: return v > 0.0f ? v : v * slope;
        case 3: return gelu<Y>(v);
        case 4: return v == -__builtin_huge_valf() ? 0.0f : silu<Y>(v);
        default: return v;
    }
}

// The epilogue of V outputs in a row from `out` on; `scale` and `bias` are theirs.
template <typename Y, bool SCALED, int V>
__device__ __forceinline__ void finish(const LinearArgs &a, int row, int out, float (&v)[V], float row_scale, const float (&scale)[V],
                                       const float (&bias)[V], const Vec<Y, V> &residual) {
    if constexpr (SCALED) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = v[e] * row_scale * scale[e];
    }
    if (a.bias != nullptr) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] += bias[e];
    }
    if (a.activation != 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = activate<Y>(v[e], a.activation, a.slope);
    }
    if (a.residual != nullptr) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] += static_cast<float>(residual[e]);
    }
    Vec<Y, V> y;
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = static_cast<Y>(v[e]);
    store_vector<false, Y, V>(static_cast<Y *>(a.y) + static_cast<size_t>(row) * a.y_stride + out, y, a.out - out);
}

template <typename Y, int V>
__device__ __forceinline__ Vec<Y, V> residual_of(const LinearArgs &a, int row, int out) {
    if (a.residual == nullptr || row >= a.rows) return Vec<Y, V>{};
    const Y *p = static_cast<const Y *>(a.residual) + static_cast<size_t>(row) * a.residual_stride + out;
    return load_vector<false, Y, V>(p, a.out - out);
}

// Four outputs in a row with all that they take.
template <typename Y, class P>
__device__ __forceinline__ void finish_quad(const LinearArgs &a, int row, int out, const typename P::Acc &sum) {
    constexpr bool SCALED = P::kScaled;
    float v[4] = {static_cast<float>(sum[0]), static_cast<float>(sum[1]), static_cast<float>(sum[2]), static_cast<float>(sum[3])};
    const int count = a.out - out;
    const Vec<Y, 4> residual = residual_of<Y, 4>(a, row, out);
    float scale[4] = {}, bias[4] = {}, row_scale = 1.0f;
    if constexpr (SCALED) {
        row_scale = a.x_scales[row];
        const Vec<float, 4> s = load_vector<false, float, 4>(a.weight_scales + out, count);
#pragma unroll
        for (int e = 0; e < 4; ++e) scale[e] = s[e];
    }
    if (a.bias != nullptr) {
        const Vec<Y, 4> b = load_vector<false, Y, 4>(static_cast<const Y *>(a.bias) + out, count);
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = static_cast<float>(b[e]);
    }
    finish<Y, SCALED, 4>(a, row, out, v, row_scale, scale, bias, residual);
}

}  // namespace bl
