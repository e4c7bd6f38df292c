// Matrix product of rows with bias, activation and residual in its epilogue:
//
//   y[i][o] = act(sum_c x[i][c] w[o][c] * (x_scales[i] w_scales[o]) + bias[o]) + residual[i][o]
#include "linear_device.h"

namespace bl {
namespace {

// Workgroup tiles: BM rows by BN outputs, WM x WN waves.
//
// ALIGNED: rows of x and weight are whole 16-byte chunks at multiples of 16 bytes and a tile's rows lie within
// 2 GB: chunks go straight to LDS, and those behind a row's end, which the buffer's range cuts off, are zeros.
// Else chunks of any alignment pass through registers.
template <class P, typename Y, int BM, int BN, int WM, int WN, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN) void linear_kernel(LinearArgs a) {
    typedef typename P::Elem E;
    constexpr int kWaves = WM * WN;
    constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements of a chunk
    constexpr int kStage = (BM + BN) * kTileBytes;
    constexpr int kLoads = (BM + BN) / 8 / kWaves;  // a wave's instructions of 8 rows each
    constexpr int NI = BN / WN / 16, NJ = BM / WM / 16;
    static_assert((BM / 8) % kWaves == 0 && (BN / 8) % kWaves == 0, "whole instructions a wave");
    __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Tile t = tile_of(a, BM, BN);
    if (t.m >= a.rows || t.first >= t.end) return;  // uniform

    const E *const x = static_cast<const E *>(a.x) + static_cast<size_t>(t.m) * a.x_stride;
    const E *const w = static_cast<const E *>(a.weight) + static_cast<size_t>(t.n) * a.weight_stride;
    const int rows = a.rows - t.m < BM ? a.rows - t.m : BM;
    const int outs = a.out - t.n < BN ? a.out - t.n : BN;

    typename P::Acc acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = {};

    // Row r of a stage holds its chunk c at place c ^ (r & 7), so that the 16 rows of a fragment fall on all banks.
    const int chunk = (lane & 7) ^ (lane >> 3);  // what this lane brings: rows 8 apart share r & 7
    unsigned offset[kLoads];
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const bool of_x = i < BM / 8 / kWaves;
            const int r = (of_x ? i * kWaves + wave : (i - BM / 8 / kWaves) * kWaves + wave) * 8 + (lane >> 3);
            const int last = (of_x ? rows : outs) - 1;
            const size_t stride = of_x ? a.x_stride : a.weight_stride;
            offset[i] = static_cast<unsigned>((r < last ? r : last) * stride * sizeof(E)) + 16u * chunk;
        }
    }
    auto issue = [&](int slot, int k0) {  // k0 in elements
        char *const base = lds + slot * kStage;
        if constexpr (ALIGNED) {
            const bool inside = k0 + chunk * kPer < a.in;
            const int kb = k0 * static_cast<int>(sizeof(E));
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const bool of_x = i < BM / 8 / kWaves;
                const int place = of_x ? i * kWaves + wave : BM / 8 + (i - BM / 8 / kWaves) * kWaves + wave;
                load_to_lds(of_x ? x : w, base + place * 1024, inside ? offset[i] : kOutOfRange, kb);
            }
        }
    };
    typedef unsigned int u4 __attribute__((ext_vector_type(4)));
    u4 held[ALIGNED ? 1 : kLoads];
    auto fetch = [&](int k0) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const bool of_x = i < BM / 8 / kWaves;
                const int r = (of_x ? i * kWaves + wave : (i - BM / 8 / kWaves) * kWaves + wave) * 8 + (lane >> 3);
                const int last = (of_x ? rows : outs) - 1;
                const int k = k0 + chunk * kPer;
                const E *p = (of_x ? x : w) + static_cast<size_t>(r < last ? r : last) * (of_x ? a.x_stride : a.weight_stride) + k;
                held[i] = __builtin_bit_cast(u4, load_vector<false, typename P::Raw, kPer>(
                                                     reinterpret_cast<const typename P::Raw *>(p), a.in - k));
            }
        }
    };
    auto put = [&](int slot) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const bool of_x = i < BM / 8 / kWaves;
                const int place = of_x ? i * kWaves + wave : BM / 8 + (i - BM / 8 / kWaves) * kWaves + wave;
                *reinterpret_cast<u4 *>(lds + slot * kStage + place * 1024 + lane * 16) = held[i];
            }
        }
    };

    const int wm = wave % WM, wn = wave / WM;
    const int fr = lane & 15, quad = lane >> 4;
    auto products = [&](int slot) {
        const char *const xs = lds + slot * kStage + (wm * (BM / WM) + fr) * kTileBytes;
        const char *const ws = lds + slot * kStage + (BM + wn * (BN / WN) + fr) * kTileBytes;
#pragma unroll
        for (int s = 0; s < P::kSlabs; ++s) {
            typename P::Frag wf[NI], xf[NJ];
#pragma unroll
            for (int i = 0; i < NI; ++i) wf[i] = P::load(ws + i * 16 * kTileBytes, s, quad, fr & 7);
#pragma unroll
            for (int j = 0; j < NJ; ++j) xf[j] = P::load(xs + j * 16 * kTileBytes, s, quad, fr & 7);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = P::mul(wf[i], xf[j], acc[i][j]);
        }
    };

    constexpr int kStep = kTileBytes / static_cast<int>(sizeof(E));
    if constexpr (ALIGNED) {
        issue(0, t.first * kStep);
        for (int kt = t.first, slot = 0; kt < t.end; ++kt, slot ^= 1) {
            meet();  // the stage has landed, and every wave is done with the other one
            if (kt + 1 < t.end) issue(slot ^ 1, (kt + 1) * kStep);
            products(slot);
        }
    } else {
        fetch(t.first * kStep);
        for (int kt = t.first, slot = 0; kt < t.end; ++kt, slot ^= 1) {
            put(slot);
            __syncthreads();  // a stage is written again two rounds on, behind the next barrier
            if (kt + 1 < t.end) fetch((kt + 1) * kStep);
            products(slot);
        }
    }

    // Outputs 4 quad .. 4 quad + 3 of a fragment's 16, row fr of its 16.
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int row = t.m + wm * (BM / WM) + j * 16 + fr;
        if (row >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int out = t.n + wn * (BN / WN) + i * 16 + 4 * quad;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(acc[i][j][e]);
            if (out >= a.out) continue;
            if (a.splits > 1) {
                store_part(a, t.split, row, out, v);
            } else {
                finish<Y, P::kScaled>(a, row, out, v);
            }
        }
    }
}

// The parts of split sums, added in order, and the epilogue.
template <typename Y, bool SCALED>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a) {
    const unsigned quads = (static_cast<unsigned>(a.out) + 3) / 4;
    const unsigned long long at = static_cast<unsigned long long>(workgroup_number()) * 256 + threadIdx.x;
    const unsigned long long row = at / quads;
    if (row >= static_cast<unsigned>(a.rows)) return;
    const int out = static_cast<int>(at - row * quads) * 4;
    float v[4] = {};
    for (int s = 0; s < a.splits; ++s) {
        const float *p = part_of(a, s, static_cast<int>(row), out);
        const Vec<float, 4> part = *reinterpret_cast<const Vec<float, 4> *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += part[e];
    }
    finish<Y, SCALED>(a, static_cast<int>(row), out, v);
}

struct Form {
    int bm, bn, splits;
};

// K steps of 128 bytes.
int steps_of(const LinearArgs &a, int size) { return (static_cast<int>((static_cast<long long>(a.in) * size + kTileBytes - 1) / kTileBytes)); }

Form form_of(const LinearArgs &a, int size, bool aligned) {
    Form f = {};
    const auto tiles = [&](int bm, int bn) {
        return ((static_cast<long long>(a.rows) + bm - 1) / bm) * ((static_cast<long long>(a.out) + bn - 1) / bn);
    };
    if (aligned && tiles(256, 256) >= 256) {
        f = {256, 256, 1};
    } else if (tiles(128, 128) >= 256) {
        f = {128, 128, 1};
    } else {
        f = {64, 64, 1};
        const int steps = steps_of(a, size);
        const long long t = tiles(64, 64);
        while (f.splits < 16 && t * f.splits * 2 <= 1024 && steps / (f.splits * 2) >= 4) f.splits *= 2;
    }
    return f;
}

template <class P, typename Y, bool ALIGNED>
hipError_t by_form(LinearArgs a, hipStream_t stream) {
    const Form f = form_of(a, sizeof(typename P::Elem), ALIGNED);
    const long long m = (static_cast<long long>(a.rows) + f.bm - 1) / f.bm, n = (static_cast<long long>(a.out) + f.bn - 1) / f.bn;
    a.splits = f.splits;
    a.steps = steps_of(a, sizeof(typename P::Elem));
    a.tiles_m = static_cast<int>(m);
    a.tiles_n = static_cast<int>(n);
    const unsigned long long blocks = static_cast<unsigned long long>(m) * n * f.splits;
    hipError_t e = hipSuccess;
    if (f.bm == 256) {
        if constexpr (ALIGNED) e = launch(linear_kernel<P, Y, 256, 256, 2, 4, ALIGNED>, blocks, 512, stream, a);
    } else if (f.bm == 128) {
        e = launch(linear_kernel<P, Y, 128, 128, 2, 2, ALIGNED>, blocks, 256, stream, a);
    } else {
        e = launch(linear_kernel<P, Y, 64, 64, 2, 2, ALIGNED>, blocks, 256, stream, a);
    }
    if (e != hipSuccess || f.splits == 1) return e;
    const unsigned long long quads = (static_cast<unsigned long long>(a.out) + 3) / 4 * static_cast<unsigned long long>(a.rows);
    return launch(linear_join_kernel<Y, P::kScaled>, (quads + 255) / 256, 256, stream, a);
}

bool aligned_rows(const LinearArgs &a, uint64_t size) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.weight) | a.x_stride * size |
                          a.weight_stride * size | static_cast<uint64_t>(a.in) * size;
    const uint64_t longest = (a.x_stride > a.weight_stride ? a.x_stride : a.weight_stride) * size;
    return bits % 16 == 0 && longest <= kBufferBytes / 512 && static_cast<uint64_t>(a.in) * size < kBufferBytes / 512;
}

template <class P, typename Y>
hipError_t by_alignment(const LinearArgs &a, hipStream_t stream) {
    return aligned_rows(a, sizeof(typename P::Elem)) ? by_form<P, Y, true>(a, stream) : by_form<P, Y, false>(a, stream);
}

template <class P>
hipError_t by_output(const LinearArgs &a, Elem type, hipStream_t stream) {
    switch (type) {
        case Elem::f32: return by_alignment<P, float>(a, stream);
        case Elem::bf16: return by_alignment<P, __bf16>(a, stream);
        default: return by_alignment<P, _Float16>(a, stream);
    }
}

hipError_t of_e4m3(const LinearArgs &a, Elem type, hipStream_t stream) {
    switch (type) {
        case Elem::f32: return by_alignment<OfE4m3Exact, float>(a, stream);
        case Elem::bf16: return by_alignment<OfE4m3, __bf16>(a, stream);
        default: return by_alignment<OfE4m3, _Float16>(a, stream);
    }
}

}  // namespace

size_t linear_scratch_bytes(const LinearArgs &a, Elem type, Eight eight) {
    if (a.rows <= 0) return 0;
    // either alignment's form splits alike: only the largest tile differs, which has no splits
    const Form f = form_of(a, eight != Eight::none ? 1 : (type == Elem::f32 ? 4 : 2), false);
    return f.splits > 1 ? static_cast<size_t>(f.splits) * a.rows * ((static_cast<size_t>(a.out) + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_linear(const LinearArgs &a, Elem type, Eight eight, hipStream_t stream) {
    if (a.rows <= 0) return hipSuccess;
    switch (eight) {
        case Eight::e4m3: return of_e4m3(a, type, stream);
        case Eight::int8: return by_output<OfInt8>(a, type, stream);
        default: break;
    }
    switch (type) {
        case Elem::f32: return by_alignment<OfF32, float>(a, stream);
        case Elem::bf16: return by_alignment<Of16<__bf16>, __bf16>(a, stream);
        default: return by_alignment<Of16<_Float16>, _Float16>(a, stream);
    }
}

}  // namespace bl
