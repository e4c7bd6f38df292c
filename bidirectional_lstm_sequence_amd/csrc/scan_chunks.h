// The chunked form of the selective state space scan on the matrix cores.
//
// Within a chunk of L rows, with cum_t the sum of the exponents D_i a up to row t and S the state
// before the chunk,
//   y_t = exp(cum_t) S c_t + sum_{s <= t} (c_t . b_s) exp(cum_t - cum_s) D_s x_s
//   S'  = exp(cum_L) S + sum_s exp(cum_L - cum_s) D_s x_s (x) b_s
// are four matrix products. One workgroup takes a head of a run of rows (a whole sequence, or a
// part of it where there are few) and walks over its chunks with the state in registers, so x, z, b
// and c are read once and y is written once. P / 16 waves; wave w owns channels 16 w .. 16 w + 15:
//   1. M[t][s] = (c_t . b_s) exp(cum_t - cum_s) D_s for s <= t: 16 x 16 blocks on and below the
//      diagonal, spread over the waves, into LDS. The others read as zeros.
//   2. y = (S C^T) exp(cum) + X^T M^T, the wave's 16 channels by L rows. The state is the left
//      operand straight from the registers that step 3 leaves it in: its accumulator layout (channel
//      = lane % 16, state 16 i + 4 (lane / 16) + r) is the operand layout of K steps whose K order
//      is (tile parity, r) within a lane group, and c is read in that order.
//   3. S' = exp(cum_L) S + B^T (w X) with w_s = exp(cum_L - cum_s) D_s; b and x are read from LDS by
//      columns (ds_read_b64_tr_b16 for 16-bit elements).
// The next chunk's rows travel from memory to registers meanwhile.
//
// Precision. Exponents are summed in float64 and kept as two floats, so a difference of two of
// them carries no more than the rounding of the difference. 16-bit inputs enter products as they
// are (fp16 as two bf16 parts, exactly). Float32 operands enter as bf16 parts, each rounding leaving
// at most 2^-8 of what it rounds: w x, whose products a state sums up over a whole sequence, in
// three parts (2^-24 left, as float32 itself), M and S, whose products only meet a 16-bit output, in
// two (2^-16 left). float32 inputs take the FP32 matrix instructions. Sums and the state are float32. Non-finite x must not reach the rows before it through a zero of
// M: where a wave's outputs hold one, it takes the products with M again, row by row.
#pragma once

#include "scan_device.h"

namespace bl {
namespace scan_chunks {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef short h4 __attribute__((ext_vector_type(4)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

struct Parts {
    b8 hi, lo;
};

struct Parts3 {
    b8 hi, mid, lo;
};

__device__ __forceinline__ f4 mfma(b8 a, b8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

__device__ __forceinline__ Parts split(const float (&v)[8]) {
    Parts p;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        p.hi[j] = static_cast<__bf16>(v[j]);
        p.lo[j] = static_cast<__bf16>(v[j] - static_cast<float>(p.hi[j]));
    }
    return p;
}

__device__ __forceinline__ Parts3 split3(const float (&v)[8]) {
    Parts3 p;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        p.hi[j] = static_cast<__bf16>(v[j]);
        const float rest = v[j] - static_cast<float>(p.hi[j]);
        p.mid[j] = static_cast<__bf16>(rest);
        p.lo[j] = static_cast<__bf16>(rest - static_cast<float>(p.mid[j]));
    }
    return p;
}

// 4 rows x 16 columns of 16-bit elements a group of 16 lanes: lane i of the group names four
// elements of row i / 4, columns 4 (i % 4), and receives column i of the four rows.
template <typename T>
__device__ __forceinline__ Vec<T, 4> column4(const T *p) {
    typedef __attribute__((address_space(3))) h4 *Lds;
    return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
}

// Operands of the products for one input type. A fragment holds 8 values of K for row (or column)
// lane % 16, K = 8 (lane / 16) + j unless read otherwise on both sides. In: values of an input tensor;
// Made: float32 values on their way to an output; Kept: to the state.
template <typename T>
struct Operand;

template <>
struct Operand<__bf16> {
    typedef b8 In;
    typedef Parts Made;
    typedef Parts3 Kept;
    typedef __bf16 Stored;
    static constexpr int kPlanes = 2;
    static __device__ __forceinline__ In rows(const __bf16 *p) { return *reinterpret_cast<const b8 *>(p); }
    static __device__ __forceinline__ In halves(const __bf16 *p, const __bf16 *q) {
        return __builtin_shufflevector(*reinterpret_cast<const b4 *>(p), *reinterpret_cast<const b4 *>(q), 0, 1, 2, 3, 4, 5,
                                       6, 7);
    }
    static __device__ __forceinline__ In columns(const __bf16 *p, int stride, int lane) {
        const __bf16 *at = p + (8 * (lane >> 4) + ((lane & 15) >> 2)) * stride + (lane & 3) * 4;
        return __builtin_shufflevector(column4(at), column4(at + 4 * stride), 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __forceinline__ float value(const In &a, int j) { return static_cast<float>(a[j]); }
    static __device__ __forceinline__ Made make(const float (&v)[8]) { return split(v); }
    static __device__ __forceinline__ Kept keep(const float (&v)[8]) { return split3(v); }
    static __device__ __forceinline__ Made stored(const __bf16 *p, int plane) {
        return {*reinterpret_cast<const b8 *>(p), *reinterpret_cast<const b8 *>(p + plane)};
    }
    static __device__ __forceinline__ void store4(__bf16 *p, int plane, const float (&v)[4]) {
        b4 hi, lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi[j] = static_cast<__bf16>(v[j]);
            lo[j] = static_cast<__bf16>(v[j] - static_cast<float>(hi[j]));
        }
        *reinterpret_cast<b4 *>(p) = hi;
        *reinterpret_cast<b4 *>(p + plane) = lo;
    }
    static __device__ __forceinline__ f4 mul(const In &a, const In &b, f4 c) { return mfma(a, b, c); }
    static __device__ __forceinline__ f4 mul(const Made &a, const In &b, f4 c) { return mfma(a.hi, b, mfma(a.lo, b, c)); }
    static __device__ __forceinline__ f4 mul(const In &a, const Made &b, f4 c) { return mfma(a, b.hi, mfma(a, b.lo, c)); }
    static __device__ __forceinline__ f4 mul(const In &a, const Kept &b, f4 c) {
        return mfma(a, b.hi, mfma(a, b.mid, mfma(a, b.lo, c)));
    }
};

template <>
struct Operand<_Float16> {
    typedef Parts In;  // exact: 8 + 8 bits hold the 11 of an fp16
    typedef Parts Made;
    typedef Parts3 Kept;
    typedef __bf16 Stored;
    static constexpr int kPlanes = 2;
    static __device__ __forceinline__ In widen(const Vec<_Float16, 8> &h) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(h[j]);
        return split(v);
    }
    static __device__ __forceinline__ In rows(const _Float16 *p) { return widen(*reinterpret_cast<const Vec<_Float16, 8> *>(p)); }
    static __device__ __forceinline__ In halves(const _Float16 *p, const _Float16 *q) {
        return widen(__builtin_shufflevector(*reinterpret_cast<const Vec<_Float16, 4> *>(p),
                                             *reinterpret_cast<const Vec<_Float16, 4> *>(q), 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ In columns(const _Float16 *p, int stride, int lane) {
        const _Float16 *at = p + (8 * (lane >> 4) + ((lane & 15) >> 2)) * stride + (lane & 3) * 4;
        return widen(__builtin_shufflevector(column4(at), column4(at + 4 * stride), 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ float value(const In &a, int j) {
        return static_cast<float>(a.hi[j]) + static_cast<float>(a.lo[j]);
    }
    static __device__ __forceinline__ Made make(const float (&v)[8]) { return split(v); }
    static __device__ __forceinline__ Kept keep(const float (&v)[8]) { return split3(v); }
    static __device__ __forceinline__ Made stored(const __bf16 *p, int plane) { return Operand<__bf16>::stored(p, plane); }
    static __device__ __forceinline__ void store4(__bf16 *p, int plane, const float (&v)[4]) {
        Operand<__bf16>::store4(p, plane, v);
    }
    // products of parts that make at most 2^-24 of the whole are left out
    static __device__ __forceinline__ f4 mul(const In &a, const Kept &b, f4 c) {
        return mfma(a.hi, b.hi, mfma(a.hi, b.mid, mfma(a.lo, b.hi, mfma(a.lo, b.mid, mfma(a.hi, b.lo, c)))));
    }
    // the product of the two small parts, at most 2^-16 of the whole, is left out
    static __device__ __forceinline__ f4 mul(const Parts &a, const Parts &b, f4 c) {
        return mfma(a.hi, b.hi, mfma(a.hi, b.lo, mfma(a.lo, b.hi, c)));
    }
};

template <>
struct Operand<float> {
    struct In {
        float v[8];
    };
    typedef In Made;
    typedef In Kept;
    typedef float Stored;
    static constexpr int kPlanes = 1;
    static __device__ __forceinline__ In halves(const float *p, const float *q) {
        In r;
        const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(q);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.v[j] = a[j];
            r.v[4 + j] = b[j];
        }
        return r;
    }
    static __device__ __forceinline__ In rows(const float *p) { return halves(p, p + 4); }
    static __device__ __forceinline__ In columns(const float *p, int stride, int lane) {
        In r;
        const float *at = p + 8 * (lane >> 4) * stride + (lane & 15);
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = at[j * stride];
        return r;
    }
    static __device__ __forceinline__ float value(const In &a, int j) { return a.v[j]; }
    static __device__ __forceinline__ Made make(const float (&v)[8]) {
        In r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = v[j];
        return r;
    }
    static __device__ __forceinline__ Kept keep(const float (&v)[8]) { return make(v); }
    static __device__ __forceinline__ Made stored(const float *p, int) { return rows(p); }
    static __device__ __forceinline__ void store4(float *p, int, const float (&v)[4]) { store_floats<float, 4>(p, v); }
    static __device__ __forceinline__ f4 mul(const In &a, const In &b, f4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
        return c;
    }
};

// 16 bytes of a row; element by element where rows are not aligned to them.
template <typename T>
__device__ __forceinline__ uint4 load16(const T *p, bool wide) {
    if (wide) return *reinterpret_cast<const uint4 *>(p);
    Vec<T, 16 / sizeof(T)> v;
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) v[i] = p[i];
    return __builtin_bit_cast(uint4, v);
}

template <typename T>
__device__ __forceinline__ void load4(const T *p, bool wide, float (&out)[4]) {
    if (wide) {
        load_floats<T, 4>(p, out);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = static_cast<float>(p[i]);
    }
}

// Rows of a chunk: 64, or 32 where the tiles of b and c would leave a CU one workgroup.
template <typename T, int N>
constexpr int chunk_rows() { return sizeof(T) == 4 || N > 128 ? 32 : 64; }

// The parts of a split sequence: run r's own end state (from a zero start; run 0 of a sequence from
// the sequence's own), [runs][heads][P][N] floats, then the log2 of its decay, [runs][heads].
// phase 0: a sequence's first run whole, and the end states of the others but the last;
// phase 1: the other runs whole, from the states that phase 0 left.
template <typename T, int P, int N>
__global__ __launch_bounds__(4 * P, 2) void scan_chunk_kernel(ScanArgs a, int run_rows, int runs, int phase, bool wide) {
    using F = Operand<T>;
    typedef typename F::Stored Stored;
    constexpr int kWaves = P / 16;
    constexpr int kThreads = 64 * kWaves;
    constexpr int L = chunk_rows<T, N>();
    constexpr int kBlocks = L / 16;           // row blocks
    constexpr int kSteps = L / 32;            // K steps over a chunk's rows
    constexpr int NP = N < 32 ? 32 : N;       // states, padded with zeros to a K step
    constexpr int kTiles = NP / 16;
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    // rows padded by 16 bytes: 16 rows' 16-byte reads then cover all banks
    constexpr int CS = NP + VE, XS = P + VE;
    constexpr int MS = L + 16 / static_cast<int>(sizeof(Stored));
    constexpr int kPlane = L * MS;
    constexpr int NV = NP / VE, PV = P / VE;
    constexpr int kBcEach = (L * NV + kThreads - 1) / kThreads;
    constexpr int kXEach = (L * PV + kThreads - 1) / kThreads;
    __shared__ __attribute__((aligned(16))) T cs[L * CS];
    __shared__ __attribute__((aligned(16))) T bs[L * CS];
    __shared__ __attribute__((aligned(16))) T xs[L * XS];
    __shared__ __attribute__((aligned(16))) Stored ms[F::kPlanes * kPlane];
    // of the chunk at hand and the next: log2 of the decay since the chunk's start (two parts), the
    // step, the decay itself, and the step times the decay to the chunk's end
    __shared__ __attribute__((aligned(16))) float cum_hi[2][L], cum_lo[2][L], steps[2][L], since[2][L], to_end[2][L];
    __shared__ float through[2];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int col = lane & 15;
    const int quad = lane >> 4;
    const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.heads));
    const int run = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.heads));
    const int j = sequence_of_run(a.seq, run, run_rows);
    const Span span = span_of(a.seq, j);
    const int first_run = run_base(a.seq, j, run_rows);
    const long long offset = static_cast<long long>(run - first_run) * run_rows;
    if (offset < 0 || offset >= span.length) return;
    const int place = a.state != nullptr ? place_of(a.seq, j) : 0;
    if (place < 0) return;
    const int rows = static_cast<int>(span.length - offset < run_rows ? span.length - offset : run_rows);
    const bool last = offset + rows == span.length;
    const bool first = offset == 0;
    if (phase == 0 ? !first && last : first) return;
    const bool whole = phase == 1 || first;

    const int g = h / (a.heads / a.groups);
    const long long row0 = span.first + offset;
    const int p_lane = 16 * wave + col;  // this lane's channel in the state
    float *cache = a.state != nullptr ? a.state + ((static_cast<size_t>(place) * a.heads + h) * P + p_lane) * N : nullptr;
    float *parts = static_cast<float *>(a.scratch);
    auto part = [&](int r) { return parts + ((static_cast<size_t>(r) * a.heads + h) * P + p_lane) * N; };
    float *totals = parts + static_cast<size_t>(runs) * a.heads * P * N;

    f4 s[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) s[i] = f4{0.f, 0.f, 0.f, 0.f};
    auto load_state = [&](const float *from, float keep) {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) s[i] = s[i] * keep + *reinterpret_cast<const f4 *>(from + 16 * i + 4 * quad);
    };
    auto store_state = [&](float *to) {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) *reinterpret_cast<f4 *>(to + 16 * i + 4 * quad) = s[i];
    };
    if (first) {
        if (cache != nullptr && !starts_fresh(a.seq, j)) load_state(cache, 0.0f);
    } else if (whole) {
        for (int r = first_run; r < run; ++r) {
            load_state(part(r), __builtin_amdgcn_exp2f(totals[static_cast<size_t>(r) * a.heads + h]));
        }
    }

    const T *xg = static_cast<const T *>(a.x) + row0 * a.x_stride + h * P;
    const T *bg = static_cast<const T *>(a.b) + row0 * a.b_stride + g * N;
    const T *cg = static_cast<const T *>(a.c) + row0 * a.c_stride + g * N;
    const T *zg = a.z != nullptr ? static_cast<const T *>(a.z) + row0 * a.z_stride + h * P : nullptr;
    T *yg = static_cast<T *>(a.y) + row0 * a.y_stride + h * P;
    const int chunks = (rows + L - 1) / L;

    // a chunk's rows on their way through registers; rows behind the run's end are zeros
    uint4 rc[kBcEach], rb[kBcEach], rx[kXEach];
    float dt_next = 0.0f;
    auto fetch = [&](int chunk) {
        const int t0 = chunk * L, n = rows - t0 < L ? rows - t0 : L;
#pragma unroll
        for (int u = 0; u < kBcEach; ++u) {
            const int at = tid + u * kThreads, t = at / NV, v = at % NV * VE;
            const bool live = t < n && v < N;  // at < L NV follows from t < n <= L
            rb[u] = live ? load16(bg + static_cast<size_t>(t0 + t) * a.b_stride + v, wide) : uint4{0, 0, 0, 0};
            if (whole) rc[u] = live ? load16(cg + static_cast<size_t>(t0 + t) * a.c_stride + v, wide) : uint4{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < kXEach; ++u) {
            const int at = tid + u * kThreads, t = at / PV, v = at % PV * VE;
            rx[u] = t < n ? load16(xg + static_cast<size_t>(t0 + t) * a.x_stride + v, wide) : uint4{0, 0, 0, 0};
        }
        if (wave == 0 && lane < n) dt_next = load_dt<T>(a, row0 + t0 + lane, h);
    };
    auto stage = [&] {
#pragma unroll
        for (int u = 0; u < kBcEach; ++u) {
            const int at = tid + u * kThreads, t = at / NV, v = at % NV * VE;
            if (L * NV % kThreads != 0 && at >= L * NV) continue;
            *reinterpret_cast<uint4 *>(bs + t * CS + v) = rb[u];
            if (whole) *reinterpret_cast<uint4 *>(cs + t * CS + v) = rc[u];
        }
#pragma unroll
        for (int u = 0; u < kXEach; ++u) {
            const int at = tid + u * kThreads, t = at / PV, v = at % PV * VE;
            if (L * PV % kThreads != 0 && at >= L * PV) continue;
            *reinterpret_cast<uint4 *>(xs + t * XS + v) = rx[u];
        }
    };
    const double exponent = static_cast<double>(a.a[h]) * 1.4426950408889634074;
    double run_total = 0.0;
    // wave 0: steps and decays of the rows fetched last; a row behind the end has step 0 and decay 1
    auto decays = [&](int chunk) {
        const int buf = chunk & 1, n = rows - chunk * L;
        const float step = lane < n && lane < L ? step_from(a, dt_next, h) : 0.0f;
        double cum = static_cast<double>(step) * exponent;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
            const double before = __shfl_up(cum, o);
            if (lane >= o) cum += before;
        }
        const double total = __shfl(cum, L - 1);
        run_total += total;
        if (lane < L) {
            const float hi = static_cast<float>(cum);
            cum_hi[buf][lane] = hi;
            cum_lo[buf][lane] = static_cast<float>(cum - static_cast<double>(hi));
            steps[buf][lane] = step;
            since[buf][lane] = __builtin_amdgcn_exp2f(hi);
            to_end[buf][lane] = step * __builtin_amdgcn_exp2f(static_cast<float>(total - cum));
        }
        if (lane == 0) through[buf] = __builtin_amdgcn_exp2f(static_cast<float>(total));
    };

    // blocks of M above the diagonal that a K step of 32 rows still reads
    for (int i = tid; i < F::kPlanes * kPlane; i += kThreads) ms[i] = static_cast<Stored>(0.0f);
    fetch(0);
    if (wave == 0) decays(0);
    const float skip = a.d != nullptr ? a.d[h] : 0.0f;
    const int p_quad = 16 * wave + 4 * quad;  // first of this lane's four channels in y

    for (int chunk = 0; chunk < chunks; ++chunk) {
        const int buf = chunk & 1;
        const int n = rows - chunk * L < L ? rows - chunk * L : L;
        __syncthreads();  // the chunk before has been read
        stage();
        __syncthreads();
        if (chunk + 1 < chunks) fetch(chunk + 1);
        if (whole) {
            float z[kBlocks][4];
            if (zg != nullptr) {
#pragma unroll
                for (int tb = 0; tb < kBlocks; ++tb) {
                    const int t = 16 * tb + col;
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[tb][e] = 0.0f;
                    if (t < n) load4(zg + static_cast<size_t>(chunk * L + t) * a.z_stride + p_quad, wide, z[tb]);
                }
            }
            // 1. M
            for (int block = wave; block < kBlocks * (kBlocks + 1) / 2; block += kWaves) {
                const int tb = block < 1 ? 0 : (block < 3 ? 1 : (block < 6 ? 2 : 3));
                const int sb = block - tb * (tb + 1) / 2;
                f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < NP / 32; ++i) {
                    acc = F::mul(F::rows(bs + (16 * sb + col) * CS + 32 * i + 8 * quad),
                                 F::rows(cs + (16 * tb + col) * CS + 32 * i + 8 * quad), acc);
                }
                const int t = 16 * tb + col;
                const float hi = cum_hi[buf][t], lo = cum_lo[buf][t];
                float m[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int sr = 16 * sb + 4 * quad + r;
                    const float d = (hi - cum_hi[buf][sr]) + (lo - cum_lo[buf][sr]);
                    m[r] = sr <= t ? acc[r] * (__builtin_amdgcn_exp2f(d) * steps[buf][sr]) : 0.0f;
                }
                F::store4(ms + t * MS + 16 * sb + 4 * quad, kPlane, m);
            }
            // 2. from the state
            f4 y[kBlocks];
            auto from_state = [&] {
#pragma unroll
                for (int tb = 0; tb < kBlocks; ++tb) y[tb] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < NP / 32; ++i) {
                    const float v[8] = {s[2 * i][0], s[2 * i][1], s[2 * i][2], s[2 * i][3],
                                        s[2 * i + 1][0], s[2 * i + 1][1], s[2 * i + 1][2], s[2 * i + 1][3]};
                    const typename F::Made left = F::make(v);
#pragma unroll
                    for (int tb = 0; tb < kBlocks; ++tb) {
                        const T *at = cs + (16 * tb + col) * CS + 32 * i + 4 * quad;
                        y[tb] = F::mul(left, F::halves(at, at + 16), y[tb]);
                    }
                }
#pragma unroll
                for (int tb = 0; tb < kBlocks; ++tb) y[tb] *= since[buf][16 * tb + col];
            };
            from_state();
            __syncthreads();  // M is whole
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const typename F::In left = F::columns(xs + 32 * k * XS + 16 * wave, XS, lane);
#pragma unroll
                for (int tb = 2 * k; tb < kBlocks; ++tb) {
                    y[tb] = F::mul(left, F::stored(ms + (16 * tb + col) * MS + 32 * k + 8 * quad, kPlane), y[tb]);
                }
            }
            float check = 0.0f;
#pragma unroll
            for (int tb = 0; tb < kBlocks; ++tb) {
#pragma unroll
                for (int r = 0; r < 4; ++r) check = fmaf(y[tb][r], 0.0f, check);
            }
            if (__any(check != 0.0f)) {
                from_state();
#pragma unroll
                for (int tb = 0; tb < kBlocks; ++tb) {
                    const int t = 16 * tb + col;
                    for (int sr = 0; sr <= t; ++sr) {
                        float m = static_cast<float>(ms[t * MS + sr]);
                        if constexpr (F::kPlanes == 2) m += static_cast<float>(ms[kPlane + t * MS + sr]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[tb][r] = fmaf(m, static_cast<float>(xs[sr * XS + p_quad + r]), y[tb][r]);
                    }
                }
            }
#pragma unroll
            for (int tb = 0; tb < kBlocks; ++tb) {
                const int t = 16 * tb + col;
                float x[4], out[4];
                load_floats<T, 4>(xs + t * XS + p_quad, x);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    out[r] = a.d != nullptr ? fmaf(skip, x[r], y[tb][r]) : y[tb][r];
                    if (zg != nullptr) out[r] *= silu<T>(z[tb][r]);
                }
                if (t < n) {
                    T *to = yg + static_cast<size_t>(chunk * L + t) * a.y_stride + p_quad;
                    if (wide) {
                        store_floats<T, 4>(to, out);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) to[r] = static_cast<T>(out[r]);
                    }
                }
            }
        }
        // 3. the state behind the chunk
        const float keep = through[buf];
#pragma unroll
        for (int i = 0; i < N / 16; ++i) s[i] *= keep;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const typename F::In x = F::columns(xs + 32 * k * XS + 16 * wave, XS, lane);
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = F::value(x, e) * to_end[buf][32 * k + 8 * quad + e];
            const typename F::Kept right = F::keep(w);
#pragma unroll
            for (int i = 0; i < N / 16; ++i) s[i] = F::mul(F::columns(bs + 32 * k * CS + 16 * i, CS, lane), right, s[i]);
        }
        if (wave == 0 && chunk + 1 < chunks) decays(chunk + 1);
    }
    if (last) {
        if (cache != nullptr) store_state(cache);
    } else if (phase == 0) {
        store_state(part(run));
        if (tid == 0) totals[static_cast<size_t>(run) * a.heads + h] = static_cast<float>(run_total);
    }
}

template <typename T, int P, int N>
hipError_t run_chunks(const ScanArgs &a, int run_rows, hipStream_t stream) {
    const long long runs = static_cast<long long>(a.seq.rows / run_rows) + a.seq.sequences;
    const long long blocks = runs * a.heads;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.b) |
                           reinterpret_cast<uintptr_t>(a.c) | reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.y);
    const size_t strides = a.x_stride | a.b_stride | a.c_stride | a.z_stride | a.y_stride;
    const bool wide = bits % 16 == 0 && strides % (16 / sizeof(T)) == 0;
    for (int phase = 0; phase < (run_rows <= a.seq.rows ? 2 : 1); ++phase) {
        hipLaunchKernelGGL((scan_chunk_kernel<T, P, N>), dim3(static_cast<unsigned>(blocks)), dim3(4 * P), 0, stream, a,
                           run_rows, static_cast<int>(runs), phase, wide);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T, int P>
hipError_t by_states(const ScanArgs &a, int run_rows, hipStream_t stream) {
    switch (a.states) {
        case 16: return run_chunks<T, P, 16>(a, run_rows, stream);
        case 32: return run_chunks<T, P, 32>(a, run_rows, stream);
        case 64: return run_chunks<T, P, 64>(a, run_rows, stream);
        case 128: return run_chunks<T, P, 128>(a, run_rows, stream);
        case 256: return run_chunks<T, P, 256>(a, run_rows, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace scan_chunks

template <typename T>
hipError_t launch_scan_chunks(const ScanArgs &a, int run_rows, hipStream_t stream) {
    switch (a.width) {
        case 32: return scan_chunks::by_states<T, 32>(a, run_rows, stream);
        case 64: return scan_chunks::by_states<T, 64>(a, run_rows, stream);
        case 128: return scan_chunks::by_states<T, 128>(a, run_rows, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace bl
