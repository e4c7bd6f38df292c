// Matrix product of rows with bias, activation and residual in its epilogue:
//
//   y[i][o] = act(sum_c x[i][c] w[o][c] * (x_scales[i] w_scales[o]) + bias[o]) + residual[i][o]
//
// Many rows: tiles whose operands go straight from memory to two stages of LDS, a step of 128 bytes of K ahead; waves
// multiply 16 x 16 blocks and pass their sums through LDS to whole lines of y. A step of 256 x 256 outputs takes 1.6 us
// on all CUs (1342 TFLOP/s bfloat16, 2840 int8, at 2.2 GHz, the matrix cores half busy; e4m3, whose codes are widened to
// bf16, 2.5), a tile's start and end 18 us. 8192 x 5120 x 5120: bfloat16 with residual 403 us (1070 TFLOP/s; the library's
// plain product 464), e4m3 with gelu 332 (1290), int8 with gelu 228 (1880), float32 by parts 2370 (181 TFLOP/s; the
// library 138). Few rows: bound by the weights' bytes, one row of 5120 x 5120 bfloat16 11.3 us (floor 10.5).
#include "linear_device.h"

namespace bl {
namespace {

// One tile of BM rows by BN outputs, WM x WN waves, K steps of 128 bytes through STAGES stages of LDS.
//
// ALIGNED: rows of x and weight are whole 16-byte chunks at multiples of 16 bytes and a tile's rows lie within
// 2 GB: chunks go straight to LDS, and those behind a row's end, which the buffer's range cuts off, are zeros.
// Else chunks of any alignment pass through registers.
template <class P, typename Y, int BM, int BN, int WM, int WN, int STAGES, bool ALIGNED>
__device__ __forceinline__ void product_of_tile(const LinearArgs &a, const Tile &t, char *lds) {
    typedef typename P::Elem E;
    constexpr int kWaves = WM * WN;
    constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements of a chunk
    constexpr int kStage = (BM + BN) * kRowBytes;
    constexpr int kXLoads = BM / 8 / kWaves, kLoads = (BM + BN) / 8 / kWaves;  // a wave's instructions of 8 rows
    constexpr int NI = BN / WN / 16, NJ = BM / WM / 16;
    constexpr int kStep = kRowBytes / static_cast<int>(sizeof(E));
    static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0, "whole instructions a wave");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (t.m >= a.rows || t.first >= t.end) return;  // uniform

    const E *const x = static_cast<const E *>(a.x) + static_cast<size_t>(t.m) * a.x_stride;
    const E *const w = static_cast<const E *>(a.weight) + static_cast<size_t>(t.n) * a.weight_stride;
    const int rows = a.rows - t.m < BM ? a.rows - t.m : BM;
    const int outs = a.out - t.n < BN ? a.out - t.n : BN;

    typename P::Acc acc[NI][NJ];

    // What this lane brings: of each instruction's rows one, the chunk that belongs at its place. Rows behind the
    // last one repeat it.
    const int load_row = lane >> 3, chunk = (lane & 7) ^ load_row;
    auto row_of = [&](int i) { return ((i < kXLoads ? i : i - kXLoads) * kWaves + wave) * 8 + load_row; };
    auto place_of = [&](int i) { return ((i < kXLoads ? i : i - kXLoads) * kWaves + wave) * 1024 + (i < kXLoads ? 0 : BM * kRowBytes); };
    unsigned offset[ALIGNED ? kLoads : 1];
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = row_of(i), last = (i < kXLoads ? rows : outs) - 1;
            const size_t stride = i < kXLoads ? a.x_stride : a.weight_stride;
            offset[i] = static_cast<unsigned>((r < last ? r : last) * stride * sizeof(E)) + 16u * chunk;
        }
    }
    auto issue = [&](int slot, int kt) {
        if constexpr (ALIGNED) {
            const int k0 = kt * kStep;
            const bool inside = k0 + chunk * kPer < a.in;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                load_to_lds(i < kXLoads ? x : w, lds + slot * kStage + place_of(i), inside ? offset[i] : kOutOfRange, kt * kRowBytes);
            }
        }
    };
    I4 held[ALIGNED ? 1 : kLoads];
    auto fetch = [&](int kt) {
        if constexpr (!ALIGNED) {
            const int k = kt * kStep + chunk * kPer;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = row_of(i), last = (i < kXLoads ? rows : outs) - 1;
                const E *p = (i < kXLoads ? x : w) + static_cast<size_t>(r < last ? r : last) * (i < kXLoads ? a.x_stride : a.weight_stride) + k;
                held[i] = __builtin_bit_cast(I4, load_vector<false, E, kPer>(p, a.in - k));
            }
        }
    };
    auto put = [&](int slot) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *reinterpret_cast<I4 *>(lds + slot * kStage + place_of(i) + lane * 16) = held[i];
        }
    };

    const int wm = wave % WM, wn = wave / WM;
    const int fr = lane & 15, quad = lane >> 4, turned = fr & 7;
    // sums[i][j] += what a stage gives for the wave's 16 outputs from 16 (first + i) and 16 rows from 16 j
    auto products = [&](int slot, auto by, int first, auto &sums) {
        typedef decltype(by) Q;
        constexpr int kOuts = sizeof(sums) / sizeof(sums[0]);
        const char *const xs = lds + slot * kStage + (wm * (BM / WM) + fr) * kRowBytes;
        const char *const ws = lds + slot * kStage + (BM + wn * (BN / WN) + 16 * first + fr) * kRowBytes;
#pragma unroll
        for (int s = 0; s < kRowBytes / Q::kSlab; ++s) {
            typename Q::Frag wf[kOuts], xf[NJ];
#pragma unroll
            for (int i = 0; i < kOuts; ++i) wf[i] = staged<Q>(ws + i * 16 * kRowBytes, s, quad, turned);
#pragma unroll
            for (int j = 0; j < NJ; ++j) xf[j] = staged<Q>(xs + j * 16 * kRowBytes, s, quad, turned);
#pragma unroll
            for (int i = 0; i < kOuts; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) sums[i][j] = Q::mul(wf[i], xf[j], sums[i][j]);
        }
    };
    auto sum_up = [&](auto by, int first, auto &sums) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int s = 0; s < STAGES - 1; ++s)
                if (t.first + s < t.end) issue(s, t.first + s);
            int slot = 0;
            for (int kt = t.first; kt < t.end; ++kt) {
                // step kt has landed, and every wave is done with the stage before it, which takes the step after the
                // STAGES - 2 that are under way
                if (kt + STAGES - 2 < t.end) {
                    meet<(STAGES - 2) * kLoads>();
                } else {
                    meet<0>();
                }
                const int ahead = slot == 0 ? STAGES - 1 : slot - 1;
                if (kt + STAGES - 1 < t.end) issue(ahead, kt + STAGES - 1);
                products(slot, by, first, sums);
                slot = slot + 1 == STAGES ? 0 : slot + 1;
            }
        } else {
            fetch(t.first);
            for (int kt = t.first, slot = 0; kt < t.end; ++kt, slot ^= 1) {
                put(slot);
                __syncthreads();  // a stage is written again two rounds on, behind the next barrier
                if (kt + 1 < t.end) fetch(kt + 1);
                products(slot, by, first, sums);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = {};
    sum_up(P{}, 0, acc);
    if constexpr (__is_same(P, OfF32Split)) {
        auto odd = [](float v) { return !(fabsf(v) < __builtin_huge_valf()); };
        bool any = false;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[i][j][e] *= P::kBack;
                    any |= odd(acc[i][j][e]);
                }
        if (__syncthreads_or(any)) {
            // sixteen outputs at a time, for the registers; sums that are finite stay as they are
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                F4 again[1][NJ] = {};
                sum_up(OfF32{}, i, again);
                meet<0>();
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (odd(acc[i][j][e])) acc[i][j][e] = again[0][j][e];
            }
        }
    }

    if (a.splits > 1) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int row = t.m + wm * (BM / WM) + 16 * j + fr, out = t.n + wn * (BN / WN) + 16 * i + 4 * quad;
                const typename P::Acc &c = acc[i][j];
                if (row < a.rows && out < a.out) *reinterpret_cast<typename P::Acc *>(part_of(a, t.split, row, out)) = c;
            }
        return;
    }
    // Through LDS, 32 rows of the wave at a time, to whole lines of 16 bytes a lane: stores of four outputs from where
    // the products leave them would fill a quarter of a line each. The loop over the lines is not unrolled: as straight
    // code the epilogue of 256 x 256 outputs was 130 KB and took 25 us to fetch.
    constexpr int W = 16 * NI, V = 16 / static_cast<int>(sizeof(Y)), kLanes = W / V, kItems = 32 * kLanes;
    constexpr int kRow = W + 4;  // floats: the padding spreads rows over the banks
    static_assert(2 * BN * 4 + kWaves * 32 * kRow * 4 <= STAGES * kStage, "the epilogue fits the stages");
    static_assert(kItems % 64 == 0 && 64 % kLanes == 0, "a lane keeps its outputs");
    meet<0>();  // every wave is done with the stages
    float *const scales = reinterpret_cast<float *>(lds), *const biases = scales + BN;
    float *const mine = biases + BN + wave * 32 * kRow;
    for (int i = tid; i < BN; i += 64 * kWaves) {
        const int out = t.n + i;
        scales[i] = P::kScaled && out < a.out ? a.weight_scales[out] : 1.0f;
        biases[i] = a.bias != nullptr && out < a.out ? static_cast<float>(static_cast<const Y *>(a.bias)[out]) : 0.0f;
    }
    __syncthreads();
    const int at = lane % kLanes * V, out = t.n + wn * (BN / WN) + at;
    float scale[V], bias[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        scale[e] = scales[wn * (BN / WN) + at + e];
        bias[e] = biases[wn * (BN / WN) + at + e];
    }
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
        // what the next line takes from memory is under way while the current one is computed
        const int last = t.m + wm * (BM / WM) + 16 * j + 32;
        int row = last - 32 + lane / kLanes;
        auto row_scale_at = [&](int r) { return P::kScaled && r < last && r < a.rows ? a.x_scales[r] : 1.0f; };
        Vec<Y, V> residual = residual_of<Y, V>(a, row, out);
        float row_scale = row_scale_at(row);
        const float *line = mine + lane / kLanes * kRow + at;
        own_lds();
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const typename P::Acc &c = acc[i][j + h];
                *reinterpret_cast<F4 *>(mine + (16 * h + fr) * kRow + 16 * i + 4 * quad) =
                    F4{static_cast<float>(c[0]), static_cast<float>(c[1]), static_cast<float>(c[2]), static_cast<float>(c[3])};
            }
        own_lds();
#pragma unroll 1
        for (; row < last; row += 64 / kLanes, line += 64 / kLanes * kRow) {
            const int next_row = row + 64 / kLanes;
            const Vec<Y, V> next = residual_of<Y, V>(a, next_row < last ? next_row : a.rows, out);
            const float next_scale = row_scale_at(next_row);
            if (row < a.rows && out < a.out) {
                float sum[V];
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] = line[e];
                finish<Y, P::kScaled, V>(a, row, out, sum, row_scale, scale, bias, residual);
            }
            residual = next;
            row_scale = next_scale;
        }
    }
}

template <class P, typename Y, int BM, int BN, int WM, int WN, int STAGES, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_kernel(LinearArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[STAGES * (BM + BN) * kRowBytes];
    const Tile t = tile_of(a, BM, BN);
    if constexpr (BM == 256) {
        if (t.halved) {
            product_of_tile<P, Y, BM / 2, BN, WM, WN, STAGES, ALIGNED>(a, t, lds);
            return;
        }
    }
    product_of_tile<P, Y, BM, BN, WM, WN, STAGES, ALIGNED>(a, t, lds);
}

// Few rows: the weights' bytes are what counts. A workgroup has 16 NI outputs of all rows, up to 16 NJ; each of its
// waves takes its share of the K steps, alone, through STAGES stages of its own, and their sums meet in LDS.
// Eight rows of 128 bytes an instruction, on their way to LDS, come faster than the 16 of 64 bytes that the matrix
// instruction takes: 52 MB in 11.0 us where those took 14.7.
constexpr int kFewWaves = 4;

template <class P, typename Y, int NI, int NJ, int STAGES, bool ALIGNED>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(LinearArgs a) {
    typedef typename P::Elem E;
    constexpr int kPer = 16 / static_cast<int>(sizeof(E)), kStep = kRowBytes / static_cast<int>(sizeof(E));
    constexpr int kRow = 16 * NI + 4, kStage = 16 * (NI + NJ) * kRowBytes, kLoads = 2 * (NI + NJ);
    __shared__ __attribute__((aligned(1024))) char lds_of_all[kFewWaves * STAGES * kStage];
    static_assert(16 * NJ * kRow * 4 <= STAGES * kStage, "a share of the sums fits the wave's stages");
    const unsigned number = workgroup_number();
    const int split = static_cast<int>(number / a.tiles_n), first_out = static_cast<int>(number % a.tiles_n) * 16 * NI;
    if (split >= a.splits) return;
    const int lane = threadIdx.x & 63, fr = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char *const lds = lds_of_all + wave * STAGES * kStage;
    const int part = split * kFewWaves + wave, parts = a.splits * kFewWaves;
    const int begin = static_cast<int>(static_cast<long long>(a.steps) * part / parts);
    const int end = static_cast<int>(static_cast<long long>(a.steps) * (part + 1) / parts);

    // what this lane brings: of each instruction's eight rows one; rows and outputs behind the last ones repeat it
    const E *const weight = static_cast<const E *>(a.weight) + static_cast<size_t>(first_out) * a.weight_stride;
    const E *const x = static_cast<const E *>(a.x);
    const int load_row = lane >> 3, chunk = (lane & 7) ^ load_row;
    size_t at[kLoads];  // elements
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const bool of_w = i < 2 * NI;
        const int r = (of_w ? i : i - 2 * NI) * 8 + load_row, last = of_w ? a.out - 1 - first_out : a.rows - 1;
        at[i] = (r < last ? r : last) * (of_w ? a.weight_stride : a.x_stride) + chunk * kPer;
    }
    auto issue = [&](int slot, int kt) {
        if constexpr (ALIGNED) {
            const bool inside = kt * kStep + chunk * kPer < a.in;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                load_to_lds(i < 2 * NI ? weight : x, lds + slot * kStage + i * 1024,
                            inside ? static_cast<unsigned>(at[i] * sizeof(E)) : kOutOfRange, kt * kRowBytes);
            }
        }
    };
    I4 held[ALIGNED ? 1 : kLoads];
    auto fetch = [&](int kt) {
        if constexpr (!ALIGNED) {
            const int k = kt * kStep;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                held[i] = __builtin_bit_cast(I4, load_vector<false, E, kPer>((i < 2 * NI ? weight : x) + at[i] + k, a.in - k - chunk * kPer));
            }
        }
    };
    typename P::Acc acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = {};
    auto products = [&](int slot) {
        const char *const ws = lds + slot * kStage + fr * kRowBytes, *const xs = ws + 16 * NI * kRowBytes;
#pragma unroll
        for (int s = 0; s < kRowBytes / P::kSlab; ++s) {
            typename P::Frag wf[NI], xf[NJ];
#pragma unroll
            for (int i = 0; i < NI; ++i) wf[i] = staged<P>(ws + i * 16 * kRowBytes, s, quad, fr & 7);
#pragma unroll
            for (int j = 0; j < NJ; ++j) xf[j] = staged<P>(xs + j * 16 * kRowBytes, s, quad, fr & 7);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = P::mul(wf[i], xf[j], acc[i][j]);
        }
    };
    if constexpr (ALIGNED) {
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            if (begin + s < end) issue(s, begin + s);
        int slot = 0;
        for (int kt = begin; kt < end; ++kt) {
            if (kt + STAGES - 2 < end) {  // step kt has landed; what follows it is under way
                meet<(STAGES - 2) * kLoads, false>();
            } else {
                meet<0, false>();
            }
            if (kt + STAGES - 1 < end) issue(slot == 0 ? STAGES - 1 : slot - 1, kt + STAGES - 1);
            products(slot);
            slot = slot + 1 == STAGES ? 0 : slot + 1;
        }
    } else {
        if (begin < end) fetch(begin);
        for (int kt = begin, slot = 0; kt < end; ++kt, slot ^= 1) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *reinterpret_cast<I4 *>(lds + slot * kStage + i * 1024 + lane * 16) = held[i];
            own_lds();
            if (kt + 1 < end) fetch(kt + 1);
            products(slot);
        }
    }
    own_lds();
    float *const shares = reinterpret_cast<float *>(lds_of_all), *const mine = reinterpret_cast<float *>(lds);
    constexpr int kShare = STAGES * kStage / 4;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            *reinterpret_cast<typename P::Acc *>(mine + (16 * j + fr) * kRow + 16 * i + 4 * quad) = acc[i][j];
        }
    __syncthreads();
    // four outputs a thread
    constexpr int kQuads = 4 * NI;
    for (int item = threadIdx.x; item < 16 * NJ * kQuads; item += 64 * kFewWaves) {
        const int row = item / kQuads, col = item % kQuads * 4, out = first_out + col;
        if (row >= a.rows || out >= a.out) continue;
        typename P::Acc v = {};
#pragma unroll
        for (int u = 0; u < kFewWaves; ++u) v += *reinterpret_cast<const typename P::Acc *>(shares + u * kShare + row * kRow + col);
        if (a.splits > 1) {
            *reinterpret_cast<typename P::Acc *>(part_of(a, split, row, out)) = v;
        } else {
            finish_quad<Y, P>(a, row, out, v);
        }
    }
}

// The parts of split sums, added in order, and the epilogue.
template <class P, typename Y>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a) {
    const unsigned quads = (static_cast<unsigned>(a.out) + 3) / 4;
    const unsigned long long at = static_cast<unsigned long long>(workgroup_number()) * 256 + threadIdx.x;
    const unsigned long long long_row = at / quads;
    if (long_row >= static_cast<unsigned>(a.rows)) return;
    const int row = static_cast<int>(long_row), out = static_cast<int>(at - long_row * quads) * 4;
    typename P::Acc v = {};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) v += *reinterpret_cast<const typename P::Acc *>(part_of(a, s, row, out));
    finish_quad<Y, P>(a, row, out, v);
}

struct Form {
    int bm, bn, splits;
};

constexpr long long kCus = 256;
constexpr int kFewRows = 32;

// Up to 32 rows the few kernel, one launch (one row of 5120 x 5120 bfloat16 11.8 us in kernels, tiles of 64 x 64 with split
// sums 11.7 and 4.4 for the join; 64 rows 17.3 where those take 16). Tiles of 256 x 256 where there is one for every CU; float32 in
// parts does not fit their registers, and rows at any element pass through too many: those take tiles of 128 x 128 where
// there are four for every CU. Else tiles of 64 x 64, which are as fast as 128 x 128 or faster there (18848 x 256 x 512
// bfloat16 16.2 us and 18.1, 2048 x 2048 x 2048 26.5 and 27.7). Sums are split up to three workgroups a CU and
// not below eight steps: 128 x 5120 x 5120 20 us with 4 splits, 26 with 2; 1111 x 777 x 999 13.5 us whole, 17.7 with 2.
Form form_of(const LinearArgs &a, int size, bool aligned) {
    const auto tiles = [&](int bm, int bn) {
        return ((static_cast<long long>(a.rows) + bm - 1) / bm) * ((static_cast<long long>(a.out) + bn - 1) / bn);
    };
    const long long steps = (static_cast<long long>(a.in) * size + kRowBytes - 1) / kRowBytes;
    if (a.rows <= kFewRows) {
        Form f = {a.rows <= 16 ? 16 : 32, a.rows <= 16 ? 16 : 32, 1};
        while (f.splits < 16 && tiles(f.bm, f.bn) * f.splits * 2 <= kCus && steps / (f.splits * 2) >= 4 * kFewWaves) f.splits *= 2;
        return f;
    }
    if (aligned && size < 4) {
        if (tiles(256, 256) >= kCus) return {256, 256, 1};
    } else if (tiles(128, 128) >= 4 * kCus) {
        return {128, 128, 1};
    }
    Form f = {64, 64, 1};
    const long long t = tiles(64, 64);
    while (f.splits < 16 && t * f.splits * 2 <= 3 * kCus && steps / (f.splits * 2) >= 8) f.splits *= 2;
    return f;
}

template <class P>
struct FewOf {
    typedef P type;
};
template <>
struct FewOf<OfF32Split> {
    typedef OfF32 type;  // bound by memory, it needs no parts
};

template <class P, typename Y, bool ALIGNED>
hipError_t by_form(LinearArgs a, hipStream_t stream) {
    const Form f = form_of(a, sizeof(typename P::Elem), ALIGNED);
    const long long m = (static_cast<long long>(a.rows) + f.bm - 1) / f.bm, n = (static_cast<long long>(a.out) + f.bn - 1) / f.bn;
    a.splits = f.splits;
    a.steps = static_cast<int>((static_cast<long long>(a.in) * sizeof(typename P::Elem) + kRowBytes - 1) / kRowBytes);
    a.tiles_m = static_cast<int>(m);
    a.tiles_n = static_cast<int>(n);
    unsigned long long blocks = static_cast<unsigned long long>(m) * n * f.splits;
    if (blocks > 0x7FFFFFFFull) return hipErrorInvalidConfiguration;
    a.whole = static_cast<int>(blocks);
    hipError_t e = hipSuccess;
    typedef typename FewOf<P>::type Few;
    if (a.rows <= kFewRows) {
        constexpr unsigned kThreads = 64 * kFewWaves;
        if (f.bm == 16) {
            e = launch(linear_few_kernel<Few, Y, 1, 1, ALIGNED ? 4 : 2, ALIGNED>, blocks, kThreads, stream, a);
        } else {
            e = launch(linear_few_kernel<Few, Y, 2, 2, ALIGNED ? 4 : 2, ALIGNED>, blocks, kThreads, stream, a);
        }
    } else if (f.bm == 256) {  // see form_of: large tiles of rows on 16 bytes, middle ones of others and of float32
        // One tile a CU at a time: where the last round has work for half of the CUs or less, its tiles are halved
        // (8192 x 5120 x 5120, two and a half rounds: 404 us, 426 with whole tiles; e4m3 339 and 382).
        const unsigned long long rest = blocks % kCus;
        if (rest <= kCus / 2) {
            a.whole = static_cast<int>(blocks - rest);
            blocks += rest;
        }
        if constexpr (ALIGNED && sizeof(typename P::Elem) < 4) e = launch(linear_kernel<P, Y, 256, 256, 2, 4, 2, ALIGNED>, blocks, 512, stream, a);
    } else if (f.bm == 128) {
        if constexpr (!ALIGNED || sizeof(typename P::Elem) == 4) e = launch(linear_kernel<P, Y, 128, 128, 2, 2, 2, ALIGNED>, blocks, 256, stream, a);
    } else {
        e = launch(linear_kernel<P, Y, 64, 64, 2, 2, 2, ALIGNED>, blocks, 256, stream, a);
    }
    if (e != hipSuccess || f.splits == 1) return e;
    const unsigned long long quads = (static_cast<unsigned long long>(a.out) + 3) / 4 * static_cast<unsigned long long>(a.rows);
    return launch(linear_join_kernel<Few, Y>, (quads + 255) / 256, 256, stream, a);
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

}  // namespace

size_t linear_scratch_bytes(const LinearArgs &a, Elem type, Eight eight) {
    if (a.rows <= 0) return 0;
    // either alignment's form splits alike: only the larger tiles differ, which have no splits
    const Form f = form_of(a, eight != Eight::none ? 1 : (type == Elem::f32 ? 4 : 2), false);
    return f.splits > 1 ? static_cast<size_t>(f.splits) * a.rows * ((static_cast<size_t>(a.out) + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_linear(const LinearArgs &a, Elem type, Eight eight, hipStream_t stream) {
    if (a.rows <= 0) return hipSuccess;
    switch (eight) {
        case Eight::e4m3: return by_output<OfE4m3>(a, type, stream);
        case Eight::int8: return by_output<OfInt8>(a, type, stream);
        default: break;
    }
    switch (type) {
        case Elem::f32: return by_alignment<OfF32Split, float>(a, stream);
        case Elem::bf16: return by_alignment<Of16<__bf16>, __bf16>(a, stream);
        default: return by_alignment<Of16<_Float16>, _Float16>(a, stream);
    }
}

}  // namespace bl
