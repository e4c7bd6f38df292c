// Log probabilities of given tokens with entropy and top alternatives.
//
//   m = max z;  s = sum e^(z - m);  w = sum e^(z - m) (z - m)
//   logprob(v) = (z_v - m) - log s;  entropy = log s - w / s
//
// About 10 instructions a logit against 2 or 4 bytes: bound by memory, every logit is read once
// (the given tokens' twice). A part (m, s, w) joins another by moving both to the larger m:
// s' = s e^d, w' = e^d (w + d s) with d = m - m'.
//
// Top alternatives are ordered by a 64-bit key: the logit's bits as an ordered whole number above,
// the token's complement below, so equal logits fall to the lowest token and no two keys are
// equal. Masked tokens (minus infinity) are never candidates: where fewer than `top` tokens are
// left, every unmasked token is in the list, so the rest of it are the lowest tokens not in it.
//
// Two forms:
//  * small vocabularies (up to kSmall): a group of 8 to 64 lanes a row, several rows a wave, the
//    row in registers, `top` rounds of a maximum over the group;
//  * others: a workgroup takes a tile of 8192 logits into registers with 16-byte loads (rows need
//    no alignment: a row's first and last vector are read element by element). A lower bound of
//    the tile's top-th logit comes from the lanes' maxima: per wave the largest 16-bit prefix
//    that `top` lanes reach, found by halving with ballots, and of those the largest of the four
//    waves. The few logits that reach it go to a list in LDS and are ranked by counting. More
//    than the list holds (a tile of equal logits) are taken by `top` rounds of a maximum. A second
//    launch joins the tiles of a row, a wave each; a row of one tile needs no second launch.
#include "sequence_device.h"

namespace bl {
namespace {

typedef unsigned long long Key;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kEach = 32;                     // logits a lane of a tile
constexpr int kTile = kThreads * kEach;       // logits of a tile
constexpr int kList = 256;                    // candidates ranked by counting
constexpr int kSmall = 1024;                  // vocabularies a group of lanes takes
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;

struct Part {
    float m, s, w;
};

// A logit below every finite one, or so far below the maximum that its weight is 0, must not
// multiply that 0 by an infinity; a NaN passes.
__device__ __forceinline__ float bounded(float d) { return d < -1e30f ? -1e30f : d; }

__device__ __forceinline__ void add_logit(Part &p, float z) {
    const float d = bounded(z - p.m);
    const float e = __builtin_amdgcn_exp2f(d * kLog2e);
    p.s += e;
    p.w = fmaf(e, d, p.w);
}

__device__ __forceinline__ Part moved(const Part &p, float m) {
    const float d = bounded(p.m - m);
    const float e = __builtin_amdgcn_exp2f(d * kLog2e);
    return {m, p.s * e, e * fmaf(d, p.s, p.w)};
}

__device__ __forceinline__ Part join(const Part &a, const Part &b) {
    const float m = fmaxf(a.m, b.m);
    const Part x = moved(a, m), y = moved(b, m);
    return {m, x.s + y.s, x.w + y.w};
}

template <int GROUP>
__device__ __forceinline__ Part join_lanes(Part p) {
#pragma unroll
    for (int o = 1; o < GROUP; o <<= 1) {
        const Part other = {__shfl_xor(p.m, o), __shfl_xor(p.s, o), __shfl_xor(p.w, o)};
        p = join(p, other);  // both sides of a pair add the same two numbers
    }
    return p;
}

// Ordered bits of a logit: larger logits have larger ones, both zeros the same, NaN the largest.
__device__ __forceinline__ unsigned ordered(float z) {
    if (z != z) return 0xFFFFFFFFu;
    const unsigned b = __float_as_uint(z + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float from_ordered(unsigned o) {
    if (o == 0xFFFFFFFFu) return __builtin_nanf("");
    return __uint_as_float((o >> 31) ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ bool masked(float z) { return z == -__builtin_huge_valf(); }

// 0 is no key: no unmasked logit has ordered bits of 0.
__device__ __forceinline__ Key key_of(float z, int token) {
    return masked(z) ? 0 : (static_cast<Key>(ordered(z)) << 32) | static_cast<unsigned>(~token);
}

__device__ __forceinline__ int token_of(Key k) { return static_cast<int>(~static_cast<unsigned>(k)); }

template <int GROUP>
__device__ __forceinline__ Key most_of_lanes(Key k) {
#pragma unroll
    for (int o = 1; o < GROUP; o <<= 1) {
        const unsigned low = __shfl_xor(static_cast<unsigned>(k), o);
        const unsigned high = __shfl_xor(static_cast<unsigned>(k >> 32), o);
        const Key other = (static_cast<Key>(high) << 32) | low;
        k = other > k ? other : k;
    }
    return k;
}

// Entry `rank` of a row's top list whose sorted keys are `keys` (0 past the last unmasked token).
template <class Keys>
__device__ __forceinline__ void write_top(const LogprobArgs &a, long long row, int rank, const Keys &keys, float m,
                                          float log_s, bool empty) {
    const Key k = keys(rank);
    long long token;
    float value = -__builtin_huge_valf();
    if (k != 0) {
        token = token_of(k);
        value = from_ordered(static_cast<unsigned>(k >> 32)) - m - log_s;
    } else {
        // the (rank - listed)-th lowest token that is not in the list: every listed token at or
        // below it moves it up by one
        int listed = 0;
        while (listed < rank && keys(listed) != 0) ++listed;
        int t = rank - listed;
        for (bool again = true; again;) {
            int below = 0;
            for (int i = 0; i < listed; ++i) below += token_of(keys(i)) <= t ? 1 : 0;
            again = t != rank - listed + below;
            t = rank - listed + below;
        }
        token = t;
        if (!empty) value = value - m - log_s;  // NaN in a row with a NaN
    }
    a.top_tokens[row * a.top + rank] = token;
    a.top_logprobs[row * a.top + rank] = value;
}

// What one row's part gives, written by `lanes` lanes; lane is this one's number.
template <typename T, class Keys>
__device__ __forceinline__ void finish_row(const LogprobArgs &a, long long row, const Part &p, int lane, int lanes,
                                           const Keys &keys) {
    const bool empty = p.s == 0.0f;  // nothing is left by the mask
    const float log_s = logf(p.s);
    const T *z = static_cast<const T *>(a.logits) + row * a.stride;
    for (int i = lane; i < a.given; i += lanes) {
        const long long token = a.tokens[row * a.given + i];
        float v = __builtin_nanf("");
        if (token >= 0 && token < a.vocabulary) {
            const float zt = static_cast<float>(z[token]);
            v = empty ? -__builtin_huge_valf() : zt - p.m - log_s;
        }
        a.logprobs[row * a.given + i] = v;
    }
    if (lane == 0) a.entropy[row] = empty ? 0.0f : log_s - p.w / p.s;
    for (int r = lane; r < a.top; r += lanes) write_top(a, row, r, keys, p.m, log_s, empty);
}

// ---- small vocabularies ------------------------------------------------------------------

template <typename T, int GROUP, int EACH>
__global__ __launch_bounds__(kThreads) void small_kernel(LogprobArgs a) {
    __shared__ Key tops[kThreads / GROUP][kMostTop];
    const int lane = threadIdx.x % GROUP;
    const int group = threadIdx.x / GROUP;
    const long long row = static_cast<long long>(blockIdx.x) * (kThreads / GROUP) + group;
    const bool live = row < a.rows;
    const T *x = static_cast<const T *>(a.logits) + (live ? row : 0) * a.stride;
    float z[EACH];
    Part p = {kLowest, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int v = i * GROUP + lane;
        z[i] = v < a.vocabulary ? static_cast<float>(x[v]) : -__builtin_huge_valf();
        p.m = fmaxf(p.m, z[i]);
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) add_logit(p, z[i]);
    p = join_lanes<GROUP>(p);
    Key last = ~static_cast<Key>(0);
    for (int r = 0; r < a.top; ++r) {
        Key best = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int v = i * GROUP + lane;
            const Key k = v < a.vocabulary ? key_of(z[i], v) : 0;
            best = k < last && k > best ? k : best;
        }
        last = most_of_lanes<GROUP>(best);
        if (lane == 0) tops[group][r] = last;
    }
    __syncthreads();
    if (live) finish_row<T>(a, row, p, lane, GROUP, [&](int r) { return tops[group][r]; });
}

// ---- tiles -------------------------------------------------------------------------------

__host__ __device__ inline size_t part_words(int top) { return 2 + static_cast<size_t>(top); }  // 64-bit words of a tile

template <typename T, bool WHOLE>
__global__ __launch_bounds__(kThreads) void tile_kernel(LogprobArgs a, int tiles) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    constexpr int kVectors = kEach / V;
    __shared__ Part parts[kWaves];
    __shared__ unsigned reach[kWaves];
    __shared__ Key list[kList];
    __shared__ Key top[kMostTop];
    __shared__ Key round[kWaves];
    __shared__ int listed;

    const int tid = threadIdx.x;
    const int wave = tid >> 6;
    const long long row = blockIdx.x / static_cast<unsigned>(tiles);
    const int tile = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles));
    const T *x = static_cast<const T *>(a.logits) + row * a.stride;
    // vector n of the row holds tokens n V - skew .. n V - skew + V - 1, 16-byte aligned
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    float z[kEach];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int first = ((tile * kVectors + i) * kThreads + tid) * V - skew;
        if (first >= 0 && first + V <= a.vocabulary) {
            const Vec<T, V> v = *reinterpret_cast<const Vec<T, V> *>(x + first);
#pragma unroll
            for (int e = 0; e < V; ++e) z[i * V + e] = static_cast<float>(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int t = first + e;
                z[i * V + e] = t >= 0 && t < a.vocabulary ? static_cast<float>(x[t]) : -__builtin_huge_valf();
            }
        }
    }
    auto token = [&](int i) { return ((tile * kVectors + i / V) * kThreads + tid) * V - skew + i % V; };

    Part p = {kLowest, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kEach; ++i) p.m = fmaxf(p.m, z[i]);
    const float lane_most = p.m;
#pragma unroll
    for (int i = 0; i < kEach; ++i) add_logit(p, z[i]);
    p = join_lanes<64>(p);
    if (tid == 0) listed = 0;
    if (tid < kMostTop) top[tid] = 0;
    if (a.top > 0) {
        // the largest prefix (sign, exponent, 7 bits) that at least `top` lanes' maxima reach
        const unsigned mine = ordered(lane_most);
        unsigned bound = 0;
#pragma unroll
        for (unsigned bit = 0x80000000u; bit >= 0x10000u; bit >>= 1) {
            if (__popcll(__ballot(mine >= (bound | bit))) >= a.top) bound |= bit;
        }
        if ((tid & 63) == 0) reach[wave] = bound;
    }
    if ((tid & 63) == 0) parts[wave] = p;
    __syncthreads();
    p = join(join(parts[0], parts[1]), join(parts[2], parts[3]));
    if (a.top > 0) {
        unsigned bound = reach[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) bound = reach[w] > bound ? reach[w] : bound;
        const float least = from_ordered(bound);  // at least kLowest: every lane's maximum is
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (!(z[i] < least) && !masked(z[i])) {
                const int at = atomicAdd(&listed, 1);
                if (at < kList) list[at] = key_of(z[i], token(i));
            }
        }
        __syncthreads();
        const int n = listed;
        if (n <= kList) {
            if (tid < n) {
                const Key mine = list[tid];
                int rank = 0;
                for (int i = 0; i < n; ++i) rank += list[i] > mine ? 1 : 0;
                if (rank < a.top) top[rank] = mine;
            }
            __syncthreads();
        } else {
            Key last = ~static_cast<Key>(0);
            for (int r = 0; r < a.top; ++r) {
                Key best = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const Key k = key_of(z[i], token(i));
                    best = k < last && k > best ? k : best;
                }
                best = most_of_lanes<64>(best);
                if ((tid & 63) == 0) round[wave] = best;
                __syncthreads();
                last = round[0];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) last = round[w] > last ? round[w] : last;
                if (tid == 0) top[r] = last;
                __syncthreads();
            }
        }
    }
    if constexpr (WHOLE) {
        finish_row<T>(a, row, p, tid, kThreads, [&](int r) { return top[r]; });
    } else {
        Key *out = static_cast<Key *>(a.scratch) + (static_cast<size_t>(row) * tiles + tile) * part_words(a.top);
        if (tid == 0) {
            out[0] = (static_cast<Key>(__float_as_uint(p.s)) << 32) | __float_as_uint(p.m);
            out[1] = __float_as_uint(p.w);
        }
        if (tid < a.top) out[2 + tid] = top[tid];
    }
}

// One wave a row joins its tiles: lane l the parts of tiles l, l + 64, ..., and in each round of
// the top list it offers the best of its tiles' first keys that are not taken yet.
template <typename T>
__global__ __launch_bounds__(64) void join_kernel(LogprobArgs a, int tiles) {
    __shared__ Key top[kMostTop];
    const int lane = threadIdx.x;
    const long long row = blockIdx.x;
    const size_t words = part_words(a.top);
    const Key *in = static_cast<const Key *>(a.scratch) + static_cast<size_t>(row) * tiles * words;
    Part p = {kLowest, 0.0f, 0.0f};
    for (int t = lane; t < tiles; t += 64) {
        const Key first = in[t * words], second = in[t * words + 1];
        p = join(p, {__uint_as_float(static_cast<unsigned>(first)), __uint_as_float(static_cast<unsigned>(first >> 32)),
                     __uint_as_float(static_cast<unsigned>(second))});
    }
    p = join_lanes<64>(p);
    Key last = ~static_cast<Key>(0);
    for (int r = 0; r < a.top; ++r) {
        Key best = 0;
        for (int t = lane; t < tiles; t += 64) {
            // a tile's keys fall, so its first one below `last` is its offer
            for (int i = 0; i < a.top; ++i) {
                const Key k = in[t * words + 2 + i];
                if (k < last) {
                    best = k > best ? k : best;
                    break;
                }
            }
        }
        last = most_of_lanes<64>(best);
        if (lane == 0) top[r] = last;
        if (last == 0) {
            if (lane > r && lane < a.top) top[lane] = 0;
            break;
        }
    }
    __syncthreads();
    finish_row<T>(a, row, p, lane, 64, [&](int r) { return top[r]; });
}

// Tiles of a row, whatever its alignment: at most 7 tokens are skipped in front.
int tiles_of(int vocabulary) { return (vocabulary + 7 + kTile - 1) / kTile; }

template <typename T, int GROUP, int EACH>
hipError_t run_small(const LogprobArgs &a, hipStream_t stream) {
    constexpr int kRows = kThreads / GROUP;
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.rows) + kRows - 1) / kRows);
    hipLaunchKernelGGL((small_kernel<T, GROUP, EACH>), dim3(blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t run(const LogprobArgs &a, hipStream_t stream) {
    if (a.vocabulary <= 8) return run_small<T, 8, 1>(a, stream);
    if (a.vocabulary <= 32) return run_small<T, 16, 2>(a, stream);
    if (a.vocabulary <= 128) return run_small<T, 32, 4>(a, stream);
    if (a.vocabulary <= 256) return run_small<T, 64, 4>(a, stream);
    if (a.vocabulary <= kSmall) return run_small<T, 64, kSmall / 64>(a, stream);
    const int tiles = tiles_of(a.vocabulary);
    const long long blocks = static_cast<long long>(a.rows) * tiles;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    if (tiles == 1) {
        hipLaunchKernelGGL((tile_kernel<T, true>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a, tiles);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((tile_kernel<T, false>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a, tiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((join_kernel<T>), dim3(static_cast<unsigned>(a.rows)), dim3(64), 0, stream, a, tiles);
    return hipGetLastError();
}

}  // namespace

size_t logprob_scratch_bytes(int rows, int vocabulary, int top) {
    if (vocabulary <= kSmall || tiles_of(vocabulary) == 1) return 0;
    return static_cast<size_t>(rows) * tiles_of(vocabulary) * part_words(top) * sizeof(Key);
}

hipError_t launch_token_logprobs(const LogprobArgs &a, Elem type, hipStream_t stream) {
    if (a.rows <= 0) return hipSuccess;
    switch (type) {
        case Elem::f32: return run<float>(a, stream);
        case Elem::bf16: return run<__bf16>(a, stream);
        default: return run<_Float16>(a, stream);
    }
}

}  // namespace bl
