// The chunked form of the selective state space scan on the matrix cores.
//
// Within a chunk of L rows, with cum_t the sum of the exponents D_i a up to row t and S the state
// before the chunk,
//   y_t = exp(cum_t) S c_t + sum_{s <= t} (c_t . b_s) exp(cum_t - cum_s) D_s x_s
//   S'  = exp(cum_L) S + sum_s exp(cum_L - cum_s) D_s x_s (x) b_s
// are four matrix products. A workgroup of four waves takes 64 CT neighbouring channels of one group
// of heads (a head or a part of one or several heads: they share b and c) over a run of rows (a whole
// sequence, or a part of it where there are few) and walks over its chunks with the state in
// registers, so x and z are read once and y is written once. Per chunk the rows of b, c and x go
// through registers, a chunk ahead, into LDS; from there each wave works alone on its 16 CT channels:
//   1. y = (S C^T) exp(cum), channels by rows, and G = B C^T for the three 16 x 16 blocks s <= t, from
//      the same fragments of c; M = G exp(cum_t - cum_s) D_s for s <= t.
//   2. S' = exp(cum_L) S + B^T (w X) with w_s = exp(cum_L - cum_s) D_s.
//   3. y += X^T M, then the skip, the gate and the store.
// Every product reads its operands in the layout that another one's result has: an accumulator
// holds rows 4 q + r of column lane % 16 (q = lane / 16), and a K step of 32 takes within lane group q
// the K values {16 e + 4 q + r, e < 2, r < 4}, on both sides. So S is the left operand of 1 as 2 leaves
// it, and G that of 3 without a pass through LDS. b and x are read by columns with
// ds_read_b64_tr_b16 (16-bit types).
//
// What bounds it. With 128 bfloat16 states a chunk of a wave is 120 matrix instructions and 920 others
// (more than half of them split float32 values into bf16 parts), with two waves a SIMD, as a wave's state and
// fragments take 250 registers: vector units busy 49 % of the time, matrix units 22 %; the rest are
// waits for the products' results and the tail of unequal runs. 24 prompts of 16384 rows
// together, 64 heads of 64 channels and 128 states: a call takes 304 us where the bytes alone take 107; in a
// trace, where no launch begins before the last one's end, end states of the runs 49 us, their join 24, the
// runs 262. One prompt of 4096 rows 90 us (bytes 22), 32 windows of 589 float32 rows, 4 heads of 64 channels
// and 64 states, 54 us (bytes 11): few workgroups, each a chain of dependent chunks.
//
// Precision. Exponents are summed in float64, within a chunk and over the chunks of a run (whose total the
// join takes in float32), and kept as two floats, so a difference of two of them carries no more than the
// rounding of the difference. 16-bit inputs enter products as they are (fp16 as two bf16 parts, exactly).
// Float32 operands, w x, M and S, enter as three bf16 parts, each rounding leaving at most 2^-8 of what it
// rounds, so 2^-24 is left as in float32 itself; of fp16's products of parts those of 2^-24 and less are
// left out. float32 inputs take the FP32 matrix instructions. Sums and the state are float32. Two parts for
// M and S would leave 2^-16 of terms that may cancel; the third costs the packed prompts 12 % (304 us,
// 270), of float16 18 % (524, 443).
// A non-finite x must not reach the rows before it through a zero of M: where a wave's outputs hold
// one, it takes step 3 again without such x and sets what follows them in their channel to NaN.
#pragma once

#include <type_traits>

#include "scan_device.h"

namespace bl {
namespace scan_chunks {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned int u2 __attribute__((ext_vector_type(2)));
typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef short h4 __attribute__((ext_vector_type(4)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

struct Parts {
    b8 hi, lo;
};

struct Parts3 {
    b8 hi, mid, lo;
};

// Rows of each run of a sequence, its last one may have fewer: as few runs as `most` rows allow, of equal
// length, as a short rest would leave its place in the launch empty.
__device__ __forceinline__ int rows_of_runs(int length, int most) {
    const unsigned rows = static_cast<unsigned>(length), top = static_cast<unsigned>(most);
    const unsigned runs = (rows + top - 1) / top;
    const unsigned each = ((rows + runs - 1) / runs + 31) / 32 * 32;
    return static_cast<int>(each < top ? each : top);
}

// Where a split sequence's runs keep their states in scratch, which is sized by the rows and not by the
// sequences. Of a sequence that starts in block `at` of run_rows rows, run k >= 1 of n has slot
// at + k - 1: as (n - 1) run_rows < its length, the block borders at + 1 .. at + n - 1 all lie inside the
// sequence, so nobody else has them. Its own old state goes to slot `kept`: of split sequences, longer than
// run_rows each, one at most starts in a block. The decay of run k stands at at + k.
struct Slots {
    int at, kept, count;
};

__device__ __forceinline__ Slots slots_of(const SequenceArgs &s, int j, int first, int run_rows) {
    const int blocks = s.rows / run_rows, at = first / run_rows;
    const bool few = s.sequences <= blocks;
    return {at, blocks + (few ? j : at), blocks + (few ? s.sequences : blocks + 1)};
}

__device__ __forceinline__ f4 mfma(b8 a, b8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// Pairs of values in bf16 (one v_cvt_pk_bf16_f32), and what the rounding left of them.
__device__ __forceinline__ unsigned int round_pair(float &a, float &b) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 pair = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    unsigned int bits = __builtin_bit_cast(unsigned int, pair);
    asm("" : "+v"(bits));  // opaque, else the compiler rounds a a second time to widen it
    a -= __uint_as_float(bits << 16);
    b -= __uint_as_float(bits & 0xFFFF0000u);
    return bits;
}

__device__ __forceinline__ b8 round_all(float (&v)[8]) {
    u4 bits;
#pragma unroll
    for (int j = 0; j < 4; ++j) bits[j] = round_pair(v[2 * j], v[2 * j + 1]);
    return __builtin_bit_cast(b8, bits);
}

__device__ __forceinline__ Parts split(float (&v)[8]) {
    const b8 hi = round_all(v);
    return {hi, round_all(v)};
}

__device__ __forceinline__ Parts3 split3(float (&v)[8]) {
    const b8 hi = round_all(v);
    const b8 mid = round_all(v);
    return {hi, mid, round_all(v)};
}

// 4 rows x 16 columns of 16-bit elements a group of 16 lanes: lane i of the group names four
// elements of row i / 4, columns 4 (i % 4), and receives column i of the four rows.
template <typename T>
__device__ __forceinline__ Vec<T, 4> column4(const T *p) {
    typedef __attribute__((address_space(3))) h4 *Lds;
    return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
}

// Place of a tile's row within its 16 rows of LDS. Rows of 16-bit elements are read in two ways: four
// values of 16 rows at a time, and four rows at a time by columns. With rows padded by 16 bytes (4 of 64
// banks), neighbouring places are 4 banks apart, right for the first; the second wants the rows of
// half a block 8 banks apart, so even places take rows 0..7 and odd ones rows 8..15.
template <typename T>
__device__ __forceinline__ constexpr int place_of_row(int t) {
    return sizeof(T) == 4 ? t : (t & ~15) | (t & 7) << 1 | (t >> 3 & 1);
}

// Operands of the products for one input type: fragments of 8 values of K for row (or column)
// lane % 16, K = 16 e + 4 (lane / 16) + r in place 4 e + r. In: values of an input tensor; Made: float32
// values. A product is a sum of terms, a matrix instruction each; callers take one term of several products
// before the next, as instructions on one accumulator wait for each other.
template <typename T>
struct Operand;

// Fragments from rows of LDS (p: the lane's row and its first value) and from columns (p: the first
// column of the tile's first row; rows lie at place_of_row).
template <typename T>
__device__ __forceinline__ Vec<T, 8> row_values(const T *p) {
    return __builtin_shufflevector(*reinterpret_cast<const Vec<T, 4> *>(p), *reinterpret_cast<const Vec<T, 4> *>(p + 16), 0,
                                   1, 2, 3, 4, 5, 6, 7);
}

template <typename T>
__device__ __forceinline__ Vec<T, 8> column_values(const T *p, int stride, int lane) {
    const T *at = p + place_of_row<T>(4 * (lane >> 4) + ((lane & 15) >> 2)) * stride + (lane & 3) * 4;
    return __builtin_shufflevector(column4(at), column4(at + 16 * stride), 0, 1, 2, 3, 4, 5, 6, 7);
}

template <>
struct Operand<__bf16> {
    typedef b8 In;
    typedef Parts3 Made;
    static __device__ __forceinline__ In rows(const __bf16 *p) { return row_values(p); }
    static __device__ __forceinline__ In columns(const __bf16 *p, int stride, int lane) {
        return column_values(p, stride, lane);
    }
    static __device__ __forceinline__ float value(const In &a, int j) { return static_cast<float>(a[j]); }
    static __device__ __forceinline__ In zero_at(In a, int j) {
        a[j] = static_cast<__bf16>(0.0f);
        return a;
    }
    static __device__ __forceinline__ Made make(float (&v)[8]) { return split3(v); }
    static constexpr int kInTerms = 1, kMadeTerms = 3;
    static __device__ __forceinline__ f4 in_term(int, const In &a, const In &b, f4 c) { return mfma(a, b, c); }
    static __device__ __forceinline__ const b8 &part(int k, const Made &a) { return k == 0 ? a.lo : (k == 1 ? a.mid : a.hi); }
    static __device__ __forceinline__ f4 made_term(int k, const Made &a, const In &b, f4 c) { return mfma(part(k, a), b, c); }
    static __device__ __forceinline__ f4 made_term(int k, const In &a, const Made &b, f4 c) { return mfma(a, part(k, b), c); }
};

template <>
struct Operand<_Float16> {
    typedef Parts In;  // exact: 8 + 8 bits hold the 11 of an fp16
    typedef Parts3 Made;
    static __device__ __forceinline__ In widen(const Vec<_Float16, 8> &h) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(h[j]);
        return split(v);
    }
    static __device__ __forceinline__ In rows(const _Float16 *p) { return widen(row_values(p)); }
    static __device__ __forceinline__ In columns(const _Float16 *p, int stride, int lane) {
        return widen(column_values(p, stride, lane));
    }
    static __device__ __forceinline__ float value(const In &a, int j) {
        return static_cast<float>(a.hi[j]) + static_cast<float>(a.lo[j]);
    }
    static __device__ __forceinline__ In zero_at(In a, int j) {
        a.hi[j] = a.lo[j] = static_cast<__bf16>(0.0f);
        return a;
    }
    static __device__ __forceinline__ Made make(float (&v)[8]) { return split3(v); }
    static constexpr int kInTerms = 4, kMadeTerms = 5;
    static __device__ __forceinline__ f4 in_term(int k, const In &a, const In &b, f4 c) {
        return mfma(k == 0 || k == 1 ? a.lo : a.hi, k == 0 || k == 2 ? b.lo : b.hi, c);
    }
    // products of parts that make at most 2^-24 of the whole are left out
    static __device__ __forceinline__ f4 made_term(int k, const In &a, const Made &b, f4 c) {
        return mfma(k == 1 || k == 3 ? a.lo : a.hi, k == 0 ? b.lo : (k == 1 || k == 2 ? b.mid : b.hi), c);
    }
    static __device__ __forceinline__ f4 made_term(int k, const Made &a, const In &b, f4 c) {
        return mfma(k == 0 ? a.lo : (k == 1 || k == 2 ? a.mid : a.hi), k == 1 || k == 3 ? b.lo : b.hi, c);
    }
};

template <>
struct Operand<float> {
    struct In {
        float v[8];
    };
    typedef In Made;
    static __device__ __forceinline__ In rows(const float *p) {
        In r;
        const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(p + 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.v[j] = a[j];
            r.v[4 + j] = b[j];
        }
        return r;
    }
    static __device__ __forceinline__ In columns(const float *p, int stride, int lane) {
        In r;
        const float *at = p + 4 * (lane >> 4) * stride + (lane & 15);
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = at[((j >> 2) * 16 + (j & 3)) * stride];
        return r;
    }
    static __device__ __forceinline__ float value(const In &a, int j) { return a.v[j]; }
    static __device__ __forceinline__ In zero_at(In a, int j) {
        a.v[j] = 0.0f;
        return a;
    }
    static __device__ __forceinline__ Made make(float (&v)[8]) {
        In r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = v[j];
        return r;
    }
    static constexpr int kInTerms = 8, kMadeTerms = 8;
    static __device__ __forceinline__ f4 in_term(int k, const In &a, const In &b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[k], b.v[k], c, 0, 0, 0);
    }
    static __device__ __forceinline__ f4 made_term(int k, const In &a, const In &b, f4 c) { return in_term(k, a, b, c); }
};

// The rows of a chunk in memory: n rows from `base` on. WIDE: 16-byte aligned rows through a buffer
// resource that ends with the last row, so that rows behind it read as zeros and are not written,
// without a branch (the caller's stride keeps 64 rows below 2^31 bytes). Else rows of any alignment.
template <typename T, bool WIDE>
struct ChunkRows {
    T *base;
    size_t stride;
    int n;
    __amdgpu_buffer_rsrc_t rsrc;

    __device__ __forceinline__ ChunkRows(const T *rows, size_t row_stride, int count, int width)
        : base(const_cast<T *>(rows)), stride(row_stride), n(count) {
        if constexpr (WIDE) {
            const unsigned bytes = static_cast<unsigned>(((count - 1) * row_stride + width) * sizeof(T));
            rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, static_cast<int>(bytes), 0x00027000);
        }
    }
    __device__ __forceinline__ int offset(int t, int v, bool live) const {
        return live ? static_cast<int>((t * static_cast<unsigned>(stride) + v) * sizeof(T)) : 0x7FFFFFF0;
    }
    __device__ __forceinline__ u4 load16(int t, int v, bool live) const {
        if constexpr (WIDE) {
            return __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset(t, v, live), 0, 0);
        } else {
            if (!live || t >= n) return u4{0, 0, 0, 0};
            return __builtin_bit_cast(u4, load_vector<false, T, 16 / sizeof(T)>(base + t * stride + v, 16 / sizeof(T)));
        }
    }
    __device__ __forceinline__ Vec<T, 4> load4(int t, int v) const {
        if constexpr (WIDE && sizeof(T) == 4) {
            return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset(t, v, true), 0, 0));
        } else if constexpr (WIDE) {
            return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_raw_buffer_load_b64(rsrc, offset(t, v, true), 0, 0));
        } else {
            if (t >= n) return Vec<T, 4>{};
            return load_vector<false, T, 4>(base + t * stride + v, 4);
        }
    }
    __device__ __forceinline__ void store4(int t, int v, Vec<T, 4> value) const {
        if constexpr (WIDE && sizeof(T) == 4) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, value), rsrc, offset(t, v, true), 0, 0);
        } else if constexpr (WIDE) {
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, value), rsrc, offset(t, v, true), 0, 0);
        } else if (t < n) {
            store_vector<false, T, 4>(base + t * stride + v, value, 4);
        }
    }
};

constexpr int kThreads = 256;

constexpr int L = 32;  // rows of a chunk: one K step of the products over rows

// Sums over each half wave of 32 lanes, up to and with each lane.
__device__ __forceinline__ double running_sum(double v) {
    auto from = [](double u, auto control) {
        const int2 w = __builtin_bit_cast(int2, u);
        return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, w.x, decltype(control)::value, 0xF, 0xF, true),
                                                    __builtin_amdgcn_update_dpp(0, w.y, decltype(control)::value, 0xF, 0xF, true)));
    };
    v += from(v, std::integral_constant<int, 0x111>{});  // row_shr 1, 2, 4, 8: zero from outside the 16 lanes
    v += from(v, std::integral_constant<int, 0x112>{});
    v += from(v, std::integral_constant<int, 0x114>{});
    v += from(v, std::integral_constant<int, 0x118>{});
    const double other = __shfl(v, (threadIdx.x & 32) + 15);
    return (threadIdx.x & 16) != 0 ? v + other : v;
}

// A lane's value for the whole wave.
__device__ __forceinline__ double lane_of(double v, int lane) {
    const int2 w = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(w.x, lane), __builtin_amdgcn_readlane(w.y, lane)));
}

// A split sequence takes three launches. Scratch holds first states of runs, [slots][heads * width][N]
// floats, then the log2 of their decays, [rows / run_rows][heads] (slots_of).
//  * scan_chunk_kernel without WHOLE: the end state of every run but a sequence's last from a zero start,
//    as the first state of the next run;
//  * scan_join_kernel: first states from the sequence's own;
//  * scan_chunk_kernel with WHOLE: all runs. Only it writes the cache, whose old states the join has
//    copied: a sequence's first and last run work at the same time.
// Sequences of one run need only the last launch.
template <typename T, int N, int CT, bool WIDE, bool WHOLE>
__global__ __launch_bounds__(kThreads, 2) void scan_chunk_kernel(ScanArgs a, int run_rows, int blocks, int items) {
    using F = Operand<T>;
    using Rows = ChunkRows<T, WIDE>;
    constexpr int NP = N < 32 ? 32 : N;       // states, padded with zeros to a K step
    constexpr int kTiles = N / 16;
    constexpr int kStates = NP / 32;          // K steps over the states
    constexpr int kChannels = 64 * CT;        // of a workgroup
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    constexpr int CS = NP + VE, XS = kChannels + VE;  // rows padded by 16 bytes (place_of_row)
    constexpr int NV = NP / VE, XV = kChannels / VE;
    constexpr int kBcEach = (L * NV + kThreads - 1) / kThreads;
    constexpr int kXEach = L * XV / kThreads;
    static_assert(L * XV % kThreads == 0, "x tile");
    __shared__ __attribute__((aligned(16))) T cs[L * CS];
    __shared__ __attribute__((aligned(16))) T bs[L * CS];
    __shared__ __attribute__((aligned(16))) T xs[L * XS];
    // each wave's own, of two chunks at hand and the next two: log2 of the decay since the chunk's start
    // (two parts), the step, the decay itself, and the step times the decay to the chunk's end
    __shared__ __attribute__((aligned(16))) float decay_tables[4][2][5][2 * L];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15;
    const int quad = lane >> 4;
    const int block = static_cast<int>(workgroup_number() % static_cast<unsigned>(blocks));
    const int run = static_cast<int>(workgroup_number() / static_cast<unsigned>(blocks));
    if (run >= items) return;
    // end states: item `run` is the run whose first state slot `run` takes, of the sequence with the border of
    // blocks behind it (slots_of)
    const int j = WHOLE ? sequence_of_run_wave(a.seq, run, run_rows)
                        : sequence_of_row_wave(a.seq, (run + 1) * run_rows - 1);
    const Span span = span_of(a.seq, j);
    if (span.length == 0) return;
    const int each = rows_of_runs(span.length, run_rows);
    const int k = run - (WHOLE ? run_base(a.seq, j, run_rows) : span.first / run_rows);  // of the sequence
    const long long offset = static_cast<long long>(k) * each;
    if (offset < 0 || offset >= span.length) return;
    const int place = a.state != nullptr ? place_of(a.seq, j) : 0;
    if (place < 0) return;
    const int rows = static_cast<int>(span.length - offset < each ? span.length - offset : each);
    const bool last = offset + rows == span.length;
    const bool first = offset == 0;
    if (!WHOLE && last) return;

    // channels: of the group, of the workgroup in it, of the wave in the workgroup
    const int group_channels = a.heads / a.groups * a.width;
    const int per_group = blocks / a.groups;
    const int g = block / per_group;
    const int in_group = block % per_group * kChannels;
    const int live_channels = group_channels - in_group < kChannels ? group_channels - in_group : kChannels;
    const int wave_channel = wave * 16 * CT;
    const bool active = wave_channel < live_channels;
    const int channel0 = g * group_channels + in_group;
    const int h = active ? (channel0 + wave_channel) / a.width : 0;
    const long long row0 = span.first + offset;
    const size_t all_channels = static_cast<size_t>(a.heads) * a.width;
    // this lane's first channel in the state; the next ct's is 16 on
    const size_t state_channel = static_cast<size_t>(channel0) + wave_channel + col;
    float *cache = a.state != nullptr ? a.state + (place * all_channels + state_channel) * N + 4 * quad : nullptr;
    float *parts = static_cast<float *>(a.scratch);
    auto part = [&](int slot) { return parts + (slot * all_channels + state_channel) * N + 4 * quad; };
    const Slots slots = slots_of(a.seq, j, span.first, run_rows);
    float *totals = parts + slots.count * all_channels * N;

    f4 s[CT][kTiles];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) s[ct][i] = f4{0.f, 0.f, 0.f, 0.f};
    }
    auto load_state = [&](const float *from) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                s[ct][i] = *reinterpret_cast<const f4 *>(from + 16 * ct * N + 16 * i);
            }
        }
    };
    auto store_state = [&](float *to) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) *reinterpret_cast<f4 *>(to + 16 * ct * N + 16 * i) = s[ct][i];
        }
    };
    if (WHOLE && active) {
        if (!first) {
            load_state(part(slots.at + k - 1));
        } else if (cache != nullptr && !starts_fresh(a.seq, j)) {
            load_state(last ? cache : part(slots.kept));
        }
    }

    const T *xg = static_cast<const T *>(a.x) + row0 * a.x_stride + channel0;
    const T *bg = static_cast<const T *>(a.b) + row0 * a.b_stride + g * N;
    const T *cg = static_cast<const T *>(a.c) + row0 * a.c_stride + g * N;
    const T *zg = a.z != nullptr ? static_cast<const T *>(a.z) + row0 * a.z_stride + channel0 : nullptr;
    T *yg = static_cast<T *>(a.y) + row0 * a.y_stride + channel0;
    const int chunks = (rows + L - 1) / L;

    const T *dt_rows = static_cast<const T *>(a.dt) + row0 * a.dt_stride + h;
    const float dt_bias = a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f;
    // a chunk's rows on their way through registers; rows behind the run's end are zeros
    u4 rc[kBcEach], rb[kBcEach], rx[kXEach];
    T dt_next = static_cast<T>(0.0f);  // as it comes: widening it would wait for it
    auto fetch = [&](int chunk) {
        const size_t t0 = static_cast<size_t>(chunk) * L;
        const int n = rows - chunk * L < L ? rows - chunk * L : L;
        const Rows b_rows(bg + t0 * a.b_stride, a.b_stride, n, N), c_rows(cg + t0 * a.c_stride, a.c_stride, n, N);
        const Rows x_rows(xg + t0 * a.x_stride, a.x_stride, n, live_channels);
#pragma unroll
        for (int u = 0; u < kBcEach; ++u) {
            const int at = tid + u * kThreads, t = at / NV, v = at % NV * VE;
            const bool live = (NP == N || v < N) && (L * NV % kThreads == 0 || t < L);
            rb[u] = b_rows.load16(t, v, live);
            if (WHOLE) rc[u] = c_rows.load16(t, v, live);
        }
#pragma unroll
        for (int u = 0; u < kXEach; ++u) {
            const int at = tid + u * kThreads, t = at / XV, v = at % XV * VE;
            rx[u] = x_rows.load16(t, v, v < live_channels);
        }
    };
    // one element of dt a lane, for two chunks
    auto fetch_dt = [&](int chunk) {
        const unsigned t = static_cast<unsigned>(chunk) * L + lane;
        if (t < static_cast<unsigned>(rows)) dt_next = dt_rows[static_cast<size_t>(t) * a.dt_stride];
    };
    auto stage = [&] {
#pragma unroll
        for (int u = 0; u < kBcEach; ++u) {
            const int at = tid + u * kThreads, t = at / NV, v = at % NV * VE;
            if (L * NV % kThreads != 0 && t >= L) continue;
            *reinterpret_cast<u4 *>(bs + place_of_row<T>(t) * CS + v) = rb[u];
            if (WHOLE) *reinterpret_cast<u4 *>(cs + place_of_row<T>(t) * CS + v) = rc[u];
        }
#pragma unroll
        for (int u = 0; u < kXEach; ++u) {
            const int at = tid + u * kThreads, t = at / XV, v = at % XV * VE;
            *reinterpret_cast<u4 *>(xs + place_of_row<T>(t) * XS + v) = rx[u];
        }
    };
    const double exponent = static_cast<double>(a.a[h]) * 1.4426950408889634074;
    double run_total = 0.0;
    // log2 of the decay over a chunk: lanes 0..31 of the even one, 32..63 of the odd one
    double totals_now = 0.0, totals_next = 0.0;
    // The state is held without the decay of the last chunks, 2^scale, until that leaves 2^-20..2^20:
    // its registers are then multiplied once for several chunks. The chunks' exponents are summed in 64
    // bits: a float32 sum of up to 20 would round each of them to 2^-20, always the same way where dt is constant.
    double scale = 0.0;
    float scale_hi = 0.0f, scale_rest = 0.0f;  // 2^scale = 2^scale_hi (1 + scale_rest)
    auto part_scale = [&] {
        scale_hi = static_cast<float>(scale);
        scale_rest = static_cast<float>(scale - static_cast<double>(scale_hi)) * 0.6931471805599453f;
    };
    auto settle_scale = [&] {
        float by = __builtin_amdgcn_exp2f(scale_hi);
        if (fabsf(scale_hi) < 150.0f) by = fmaf(by, scale_rest, by);  // else 0 or infinite, with no rest to speak of
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) s[ct][i] *= by;
        }
        scale = 0.0;
        scale_hi = scale_rest = 0.0f;
    };
    // steps and decays of the two chunks whose dt came last; a row behind the end has step 0 and decay 1
    auto decays = [&](int chunk) {
        float *table = &decay_tables[wave][chunk >> 1 & 1][0][0];
        const float step = static_cast<unsigned>(chunk) * L + lane < static_cast<unsigned>(rows) ? step_from(static_cast<float>(dt_next), dt_bias, a.softplus) : 0.0f;
        const double cum = running_sum(static_cast<double>(step) * exponent);
        const double total = __shfl(cum, lane | 31);
        const float hi = static_cast<float>(cum);
        table[lane] = hi;
        table[2 * L + lane] = static_cast<float>(cum - static_cast<double>(hi));
        table[4 * L + lane] = step;
        table[6 * L + lane] = __builtin_amdgcn_exp2f(hi);
        table[8 * L + lane] = step * __builtin_amdgcn_exp2f(static_cast<float>(total - cum));
        run_total += total;  // lane 0: of even chunks, lane 32: of odd ones
        return total;
    };

    fetch(0);
    if (active) {
        fetch_dt(0);
        totals_next = decays(0);
        fetch_dt(2);
    }
    const float skip = a.d != nullptr ? a.d[h] : 0.0f;
    const int y_channel = wave_channel + 4 * quad;  // of this lane's four in y, for ct 0

    const bool gated = WHOLE && zg != nullptr;
    for (int chunk = 0; chunk < chunks; ++chunk) {
        const int n = rows - chunk * L < L ? rows - chunk * L : L;
        __syncthreads();  // the chunk before has been read
        stage();
        __syncthreads();
        if (active && (chunk & 1) == 0) {
            // before the next rows are asked for: dt came before the rows just staged, and a wait for it
            // must not become one for them
            totals_now = totals_next;
            totals_next = decays(chunk + 2);
            fetch_dt(chunk + 4);
        }
        if (chunk + 1 < chunks) fetch(chunk + 1);
        if (!active) continue;
        const float *cum_hi = &decay_tables[wave][chunk >> 1 & 1][0][0] + (chunk & 1) * L, *cum_lo = cum_hi + 2 * L,
                    *steps = cum_hi + 4 * L, *since = cum_hi + 6 * L, *to_end = cum_hi + 8 * L;
        const double total = lane_of(totals_now, (chunk & 1) * 32);
        const size_t t0 = static_cast<size_t>(chunk) * L;
        Vec<T, 4> z[2][CT];
        f4 y[2][CT], gram[3];  // blocks (s, t) = (0, 0), (0, 1), (1, 1)
        float state_decay = __builtin_amdgcn_exp2f(scale_hi);
        state_decay = fmaf(state_decay, scale_rest, state_decay);
        // behind the chunk; long before its use, as it is a chain of dependent instructions
        scale += total;
        part_scale();
        const bool settles = !(fabsf(scale_hi) < 20.0f);
        float unscaled = __builtin_amdgcn_exp2f(-scale_hi);
        unscaled = fmaf(unscaled, -scale_rest, unscaled);
        if (gated) {
            const Rows z_rows(zg + t0 * a.z_stride, a.z_stride, n, live_channels);
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) z[tb][ct] = z_rows.load4(16 * tb + col, y_channel + 16 * ct);
            }
        }
        // 1. from the state, and G
        if constexpr (WHOLE) {
#pragma unroll
            for (int k = 0; k < 3; ++k) gram[k] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) y[0][ct] = y[1][ct] = f4{0.f, 0.f, 0.f, 0.f};
            const T *at = cs + place_of_row<T>(col) * CS + 4 * quad, *bt = bs + place_of_row<T>(col) * CS + 4 * quad;
            typename F::In c[2][2], b[2][2];  // of this K step and the next, on their way early
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                c[0][k] = F::rows(at + 16 * k * CS);
                b[0][k] = F::rows(bt + 16 * k * CS);
            }
#pragma unroll
            for (int i = 0; i < kStates; ++i) {
                if (i + 1 < kStates) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        c[(i + 1) & 1][k] = F::rows(at + 16 * k * CS + 32 * (i + 1));
                        b[(i + 1) & 1][k] = F::rows(bt + 16 * k * CS + 32 * (i + 1));
                    }
                }
                const typename F::In(&cn)[2] = c[i & 1], (&bn)[2] = b[i & 1];
                typename F::Made left[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = e < 4 || kTiles > 1 ? s[ct][(2 * i + (e >> 2)) % kTiles][e & 3] : 0.0f;
                    left[ct] = F::make(v);
                }
#pragma unroll
                for (int k = 0; k < F::kInTerms; ++k) {
                    gram[0] = F::in_term(k, bn[0], cn[0], gram[0]);
                    gram[1] = F::in_term(k, bn[0], cn[1], gram[1]);
                    gram[2] = F::in_term(k, bn[1], cn[1], gram[2]);
                }
#pragma unroll
                for (int k = 0; k < F::kMadeTerms; ++k) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
                        for (int tb = 0; tb < 2; ++tb) y[tb][ct] = F::made_term(k, left[ct], cn[tb], y[tb][ct]);
                    }
                }
            }
        }
        typename F::Made m[2];
        if constexpr (WHOLE) {
            float s_hi[2][4], s_lo[2][4], s_step[2][4];
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                load_floats<float, 4>(cum_hi + 16 * sb + 4 * quad, s_hi[sb]);
                load_floats<float, 4>(cum_lo + 16 * sb + 4 * quad, s_lo[sb]);
                load_floats<float, 4>(steps + 16 * sb + 4 * quad, s_step[sb]);
            }
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const float hi = cum_hi[16 * tb + col], lo = cum_lo[16 * tb + col], decay = since[16 * tb + col] * state_decay;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int sb = e >> 2, r = e & 3;
                    v[e] = 0.0f;
                    if (sb > tb) continue;
                    const float d = (hi - s_hi[sb][r]) + (lo - s_lo[sb][r]);
                    const float full = gram[sb + tb][r] * (__builtin_amdgcn_exp2f(d) * s_step[sb][r]);
                    v[e] = sb < tb || 4 * quad + r <= col ? full : 0.0f;
                }
                m[tb] = F::make(v);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[tb][ct] *= decay;
            }
        }
        if (settles) {
            settle_scale();
            unscaled = 1.0f;
        }
        __builtin_amdgcn_sched_barrier(0);  // the registers do not hold more at once
        // 2. the state behind the chunk
        typename F::In x[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) x[ct] = F::columns(xs + wave_channel + 16 * ct, XS, lane);
        {
            typename F::Made right[CT];
            float weight[2][4];
            load_floats<float, 4>(to_end + 4 * quad, weight[0]);
            load_floats<float, 4>(to_end + 16 + 4 * quad, weight[1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) weight[e >> 2][e & 3] *= unscaled;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = F::value(x[ct], e) * weight[e >> 2][e & 3];
                right[ct] = F::make(w);
            }
            constexpr int kPair = kTiles < 2 ? 1 : 2;
            typename F::In left[2][kPair];
#pragma unroll
            for (int k = 0; k < kPair; ++k) left[0][k] = F::columns(bs + 16 * k, CS, lane);
#pragma unroll
            for (int i = 0; i < kTiles / kPair; ++i) {
                if (i + 1 < kTiles / kPair) {
#pragma unroll
                    for (int k = 0; k < kPair; ++k) left[(i + 1) & 1][k] = F::columns(bs + 16 * (kPair * (i + 1) + k), CS, lane);
                }
#pragma unroll
                for (int term = 0; term < F::kMadeTerms; ++term) {
#pragma unroll
                    for (int k = 0; k < kPair; ++k) {
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) {
                            s[ct][kPair * i + k] = F::made_term(term, left[i & 1][k], right[ct], s[ct][kPair * i + k]);
                        }
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // 3. from the chunk's own rows
        if constexpr (WHOLE) {
            f4 sums[2][CT];
            float check = 0.0f;
#pragma unroll
            for (int k = 0; k < F::kMadeTerms; ++k) {
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) sums[tb][ct] = F::made_term(k, x[ct], m[tb], k == 0 ? y[tb][ct] : sums[tb][ct]);
                }
            }
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const f4 &v = sums[tb][ct];
                    check += (v[0] + v[1]) + (v[2] + v[3]);
                }
            }
            if (__any(check * 0.0f != 0.0f)) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    // the first row of this lane's channel (16 ct + col) whose x is not finite
                    int bad = L;
                    typename F::In sound = x[ct];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (F::value(x[ct], e) * 0.0f == 0.0f) continue;
                        const int row = 16 * (e >> 2) + 4 * quad + (e & 3);
                        bad = row < bad ? row : bad;
                        sound = F::zero_at(sound, e);
                    }
                    bad = min(bad, __shfl_xor(bad, 16));
                    bad = min(bad, __shfl_xor(bad, 32));
#pragma unroll
                    for (int tb = 0; tb < 2; ++tb) {
                        sums[tb][ct] = y[tb][ct];
#pragma unroll
                        for (int k = 0; k < F::kMadeTerms; ++k) sums[tb][ct] = F::made_term(k, sound, m[tb], sums[tb][ct]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (16 * tb + col >= __shfl(bad, 4 * quad + r)) sums[tb][ct][r] = __builtin_nanf("");
                        }
                    }
                }
            }
            const Rows y_rows(yg + t0 * a.y_stride, a.y_stride, n, live_channels);
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const int t = 16 * tb + col;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const Vec<T, 4> xv =
                        *reinterpret_cast<const Vec<T, 4> *>(xs + place_of_row<T>(t) * XS + y_channel + 16 * ct);
                    Vec<T, 4> out;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        // without d the skip is 0 x, which is 0: rows whose x is not finite are not either
                        float v = fmaf(skip, static_cast<float>(xv[r]), sums[tb][ct][r]);
                        if (gated) v *= silu<T>(static_cast<float>(z[tb][ct][r]));
                        out[r] = static_cast<T>(v);
                    }
                    y_rows.store4(t, y_channel + 16 * ct, out);
                }
            }
        }
    }
    if (!active) return;
    settle_scale();
    if constexpr (WHOLE) {
        if (last && cache != nullptr) store_state(cache);
    } else {
        store_state(part(slots.at + k));
        run_total += __shfl_xor(run_total, 32);
        if (lane == 0 && (channel0 + wave_channel) % a.width == 0) {
            totals[static_cast<size_t>(slots.at + k) * a.heads + h] = static_cast<float>(run_total);
        }
    }
}

// One lane a channel and four states of a sequence: its state, then for each run but the last
// s = decay * s + the run's own end state, each the next run's first state. The parts of kAhead runs are on
// their way at once. From a zero start nothing changes up to the second run.
inline __global__ __launch_bounds__(kThreads) void scan_join_kernel(ScanArgs a, int run_rows, int lanes, int items) {
    constexpr int kAhead = 8;
    const int each = static_cast<int>((static_cast<long long>(lanes) + kThreads - 1) / kThreads);
    const int item = static_cast<int>(workgroup_number() / static_cast<unsigned>(each));
    const int at = static_cast<int>(workgroup_number() % static_cast<unsigned>(each)) * kThreads + threadIdx.x;
    if (item >= items) return;
    // few sequences: each; else, in each block of rows, the last one that starts there: no other can be split
    int j = item;
    const bool few = a.seq.sequences <= a.seq.rows / run_rows;
    if (!few) {
        const long long end = (static_cast<long long>(item) + 1) * run_rows;
        j = sequence_of_row_wave(a.seq, static_cast<int>(end < a.seq.rows ? end : a.seq.rows) - 1);
    }
    const Span span = span_of(a.seq, j);
    if (span.length == 0 || (!few && span.first / run_rows != item)) return;
    const int count = (span.length - 1) / rows_of_runs(span.length, run_rows);  // runs before the last one
    const int place = a.state != nullptr ? place_of(a.seq, j) : 0;
    if (at >= lanes || count < 1 || place < 0) return;
    const bool kept = a.state != nullptr && !starts_fresh(a.seq, j);
    const Slots slots = slots_of(a.seq, j, span.first, run_rows);
    const size_t run_floats = static_cast<size_t>(lanes) * 4;
    f4 *all = reinterpret_cast<f4 *>(a.scratch) + at;
    f4 *parts = all + static_cast<size_t>(slots.at) * lanes;  // of the runs from the second on
    const float *totals = static_cast<const float *>(a.scratch) + slots.count * run_floats +
                          static_cast<size_t>(slots.at) * a.heads + at / (a.width * a.states / 4);
    f4 s = {0.f, 0.f, 0.f, 0.f};
    if (kept) all[static_cast<size_t>(slots.kept) * lanes] = s = reinterpret_cast<const f4 *>(a.state + place * run_floats)[at];
    for (int r0 = 0; r0 < count; r0 += kAhead) {
        f4 own[kAhead];
        float decay[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i < count ? r0 + i : count - 1;
            own[i] = parts[static_cast<size_t>(r) * lanes];
            decay[i] = totals[static_cast<size_t>(r) * a.heads];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (r0 + i >= count) break;
            if (!kept && r0 + i == 0) {
                s = own[i];
            } else {
                s = s * __builtin_amdgcn_exp2f(decay[i]) + own[i];
                parts[static_cast<size_t>(r0 + i) * lanes] = s;
            }
        }
    }
}

template <typename T, int N, int CT, bool WIDE>
hipError_t run_chunks(const ScanArgs &a, int run_rows, hipStream_t stream) {
    const int group_channels = a.heads / a.groups * a.width;
    const int blocks = a.groups * ((group_channels + 64 * CT - 1) / (64 * CT));
    const int splits = a.seq.rows / run_rows, runs = splits + a.seq.sequences;
    const int lanes = a.heads * a.width * (N / 4), lane_blocks = (lanes + kThreads - 1) / kThreads;
    const int joined = a.seq.sequences <= splits ? a.seq.sequences : splits + 1;
    auto times = [](int m, int n) { return static_cast<unsigned long long>(m) * static_cast<unsigned>(n); };
    if (times(runs, blocks) > kMostWorkgroups) return hipErrorInvalidConfiguration;  // before anything has run
    if (splits > 0) {
        hipError_t e = launch(scan_chunk_kernel<T, N, CT, WIDE, false>, times(splits, blocks), kThreads, stream, a, run_rows, blocks,
                              splits);
        if (e == hipSuccess) e = launch(scan_join_kernel, times(joined, lane_blocks), kThreads, stream, a, run_rows, lanes, joined);
        if (e != hipSuccess) return e;
    }
    return launch(scan_chunk_kernel<T, N, CT, WIDE, true>, times(runs, blocks), kThreads, stream, a, run_rows, blocks, runs);
}

template <typename T, int N>
hipError_t by_alignment(ScanArgs a, int run_rows, hipStream_t stream) {
    // Two tiles of channels a wave read the fragments of b and c half as often, but 256 states of them
    // leave 16-bit types no registers for the rest. 24 sequences of 683 rows, 64 heads of 64 channels,
    // with one and two: 128 states 266 and 223 us in bfloat16, 462 and 380 in float16, 631 and 548 in float32;
    // 256 states 391 and 696, 852 and 993, 1323 and 998; 64 states 197 and 195, 311 and 231, 366 and 325.
    constexpr int CT = N > 128 && sizeof(T) == 2 ? 1 : 2;
    if (a.seq.rows == 1) {  // a single row's strides say nothing
        a.x_stride = a.y_stride = a.z_stride = static_cast<size_t>(a.heads) * a.width;
        a.b_stride = a.c_stride = static_cast<size_t>(a.groups) * a.states;
    }
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.b) |
                           reinterpret_cast<uintptr_t>(a.c) | reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.y);
    const size_t strides = a.x_stride | a.b_stride | a.c_stride | a.z_stride | a.y_stride;
    // loads element by element: 391 -> 404 us at those 256 bfloat16 states, 225 -> 247 at 128
    const bool wide = bits % 16 == 0 && strides % (16 / sizeof(T)) == 0 && strides < (1u << 22);
    return wide ? run_chunks<T, N, CT, true>(a, run_rows, stream) : run_chunks<T, N, CT, false>(a, run_rows, stream);
}

}  // namespace scan_chunks

template <typename T>
hipError_t launch_scan_chunks(const ScanArgs &a, int run_rows, hipStream_t stream) {
    switch (a.states) {
        case 16: return scan_chunks::by_alignment<T, 16>(a, run_rows, stream);
        case 32: return scan_chunks::by_alignment<T, 32>(a, run_rows, stream);
        case 64: return scan_chunks::by_alignment<T, 64>(a, run_rows, stream);
        case 128: return scan_chunks::by_alignment<T, 128>(a, run_rows, stream);
        case 256: return scan_chunks::by_alignment<T, 256>(a, run_rows, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace bl
