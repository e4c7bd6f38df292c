// Device helpers of the matrix product: operands of its element types, tiles and the epilogue.
#pragma once

#include "tile_device.h"

namespace bl {

constexpr int kTileBytes = 128;  // of one row's K step

typedef float F4 __attribute__((ext_vector_type(4)));
typedef int I4 __attribute__((ext_vector_type(4)));
typedef int I8 __attribute__((ext_vector_type(8)));

// Operands by element type. A fragment holds, for row lane % 16 of 16, what lane / 16 contributes to K; as both
// operands number K alike, any share of a row's chunks will do. `place` is the row's number modulo 8.
template <typename T>
struct Of16 {
    typedef T Elem;
    typedef T Raw;
    typedef Vec<T, 8> Frag;
    typedef F4 Acc;
    static constexpr int kSlabs = 2;
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ Frag load(const char *row, int slab, int quad, int place) {
        return *reinterpret_cast<const Frag *>(row + (((slab * 4 + quad) ^ place) * 16));
    }
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
    typedef float Raw;
    typedef F4 Frag;
    typedef F4 Acc;
    static constexpr int kSlabs = 2;
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ Frag load(const char *row, int slab, int quad, int place) {
        return *reinterpret_cast<const Frag *>(row + (((slab * 4 + quad) ^ place) * 16));
    }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, Acc c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

// e4m3 by the instruction with block scales, here 2^0, at twice the rate of 16 bits. The matrix cores bring eight
// neighbouring products of 8-bit floats to the place of the largest and drop what lies below 2^-13 of it (also
// without scales, measured; further sums are those of float32): at most 2^-10 of that product for the eight, where
// the codes themselves are within 2^-4 of what they stand for. So this one is for outputs of 16 bits.
struct OfE4m3 {
    typedef unsigned char Elem;
    typedef unsigned char Raw;
    typedef I8 Frag;
    typedef F4 Acc;
    static constexpr int kSlabs = 1;
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ Frag load(const char *row, int, int quad, int place) {
        const I4 low = *reinterpret_cast<const I4 *>(row + ((quad ^ place) * 16));
        const I4 high = *reinterpret_cast<const I4 *>(row + (((quad + 4) ^ place) * 16));
        return __builtin_shufflevector(low, high, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, const Acc &c) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
    }
};

// For outputs of 32 bits e4m3 is widened to bf16, exactly.
struct OfE4m3Exact {
    typedef unsigned char Elem;
    typedef unsigned char Raw;
    struct Frag {
        Vec<__bf16, 8> part[2];
    };
    typedef F4 Acc;
    static constexpr int kSlabs = 2;
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ Frag load(const char *row, int slab, int quad, int place) {
        const I4 codes = *reinterpret_cast<const I4 *>(row + (((slab * 4 + quad) ^ place) * 16));
        Frag f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const auto low = __builtin_amdgcn_cvt_pk_f32_fp8(codes[e], false), high = __builtin_amdgcn_cvt_pk_f32_fp8(codes[e], true);
            const int at = e % 2 * 4;
            f.part[e / 2][at] = static_cast<__bf16>(low[0]);
            f.part[e / 2][at + 1] = static_cast<__bf16>(low[1]);
            f.part[e / 2][at + 2] = static_cast<__bf16>(high[0]);
            f.part[e / 2][at + 3] = static_cast<__bf16>(high[1]);
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
    typedef unsigned char Raw;
    typedef I4 Frag;
    typedef I4 Acc;
    static constexpr int kSlabs = 2;
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ Frag load(const char *row, int slab, int quad, int place) {
        return *reinterpret_cast<const Frag *>(row + (((slab * 4 + quad) ^ place) * 16));
    }
    static __device__ __forceinline__ Acc mul(const Frag &a, const Frag &b, const Acc &c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
};

// A workgroup's tile: first row and output, and its share first .. end - 1 of the K steps.
struct Tile {
    int m, n, first, end, split;
};

// Workgroups go to the 8 XCDs in turn. Each XCD takes a range of tiles in a row, eight row tiles by all outputs
// at a time, so that what its L2 holds is used by several of its CUs.
__device__ __forceinline__ Tile tile_of(const LinearArgs &a, int bm, int bn) {
    const unsigned total = static_cast<unsigned>(a.tiles_m) * a.tiles_n;
    unsigned number = workgroup_number();
    const unsigned split = number / total;
    number -= split * total;
    const unsigned per = total / 8, rest = total % 8, xcd = number % 8, at = number / 8;
    const unsigned t = xcd * per + (xcd < rest ? xcd : rest) + at;
    constexpr unsigned kGroup = 8;
    const unsigned wide = kGroup * a.tiles_n, group = t / wide, inside = t - group * wide;
    const unsigned left = a.tiles_m - group * kGroup, high = left < kGroup ? left : kGroup;
    Tile tile;
    tile.split = static_cast<int>(split);
    if (split >= static_cast<unsigned>(a.splits)) {
        tile.m = a.rows;  // a number behind the last one
        tile.n = tile.first = tile.end = 0;
        return tile;
    }
    tile.m = static_cast<int>(group * kGroup + inside % high) * bm;
    tile.n = static_cast<int>(inside / high) * bn;
    tile.first = static_cast<int>(static_cast<long long>(a.steps) * split / a.splits);
    tile.end = static_cast<int>(static_cast<long long>(a.steps) * (split + 1) / a.splits);
    return tile;
}

__device__ __forceinline__ float *part_of(const LinearArgs &a, int split, int row, int out) {
    const size_t width = (static_cast<size_t>(a.out) + 3) / 4 * 4;
    return a.scratch + (static_cast<size_t>(split) * a.rows + row) * width + out;
}

__device__ __forceinline__ void store_part(const LinearArgs &a, int split, int row, int out, const float (&v)[4]) {
    *reinterpret_cast<F4 *>(part_of(a, split, row, out)) = F4{v[0], v[1], v[2], v[3]};
}

__device__ __forceinline__ float activate(float v, int kind, float slope) {
    switch (kind) {
        case 1: return __builtin_elementwise_maximum(v, 0.0f);
        case 2: return v > 0.0f ? v : v * slope;
        case 3: return 0.5f * v * erfcf(v * -0.7071067811865476f);  // 1 + erf, without its cancellation
        case 4: return silu<float>(v);
        default: return v;
    }
}

// The epilogue of four outputs in a row from `out` on.
template <typename Y, bool SCALED>
__device__ __forceinline__ void finish(const LinearArgs &a, int row, int out, float (&v)[4]) {
    const int count = a.out - out;
    if constexpr (SCALED) {
        const float xs = a.x_scales[row];
        const Vec<float, 4> ws = load_vector<false, float, 4>(a.weight_scales + out, count);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = v[e] * xs * ws[e];
    }
    if (a.bias != nullptr) {
        const Vec<Y, 4> b = load_vector<false, Y, 4>(static_cast<const Y *>(a.bias) + out, count);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += static_cast<float>(b[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = activate(v[e], a.activation, a.slope);
    if (a.residual != nullptr) {
        const Y *p = static_cast<const Y *>(a.residual) + static_cast<size_t>(row) * a.residual_stride + out;
        const Vec<Y, 4> r = load_vector<false, Y, 4>(p, count);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += static_cast<float>(r[e]);
    }
    Vec<Y, 4> y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = static_cast<Y>(v[e]);
    store_vector<false, Y, 4>(static_cast<Y *>(a.y) + static_cast<size_t>(row) * a.y_stride + out, y, count);
}

}  // namespace bl
