// Log probabilities of given tokens with entropy and top alternatives.
//
//   m = max z;  s = sum e^(z - m);  w = sum e^(z - m) (z - m)
//   logprob(v) = (z_v - m) - log s;  entropy = log s - w / s
//
// About 10 instructions a logit against 2 or 4 bytes; every logit is read once (the given tokens'
// twice). 512 rows of 100003 bfloat16 logits with 8 alternatives take 33 us, 3.1 TB/s, float16 ones 34,
// float32 ones 40 us, 5.2 TB/s: the instructions and the loads take about as long there and overlap in part.
// 18848 rows of 7 take 3.8 us, bound by the launch. A part (m, s, w) joins another by moving both to the larger m:
// s' = s e^d, w' = e^d (w + d s) with d = m - m'.
//
// Top alternatives are ordered by a 64-bit key: the logit's bits as an ordered whole number above,
// the token's complement below, so equal logits fall to the lowest token and no two keys are
// equal. Masked tokens (minus infinity) are never candidates: where fewer than `top` tokens are
// left, every unmasked token is in the list, so the rest of it are the lowest tokens not in it.
//
// Two forms:
//  * small vocabularies (is_small): a group of 8 to 64 lanes a row, several rows a wave, the
//    row in registers, `top` rounds of a maximum over the group and the first token that has it;
//  * others: a workgroup takes a tile of 16384 16-bit or 8192 float32 logits into registers with
//    16-byte loads (rows need no alignment: a row's first and last vector are read element by
//    element). A wave finds its maximum first, so that every logit takes one exponential. A lower
//    bound of the tile's top-th logit comes from the lanes' maxima: per wave the largest 16-bit
//    prefix that `top` lanes reach, found by halving with ballots, and of those the largest of the
//    four waves. The few logits that reach it go to a list in LDS and are ranked by counting. More
//    than the list holds (a tile of equal logits) are taken by `top` rounds of a maximum. A second
//    launch joins the tiles of a row, a workgroup each; a row of one tile needs no second launch.
#include <type_traits>

#include "sequence_device.h"

namespace bl {
namespace {

typedef unsigned long long Key;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kList = 256;                    // candidates ranked by counting
constexpr int kMostTiles = 129;               // 2^20 float32 logits and a vector's skew
constexpr int kSmall = 1024;                  // vocabularies a group of lanes takes (is_small)
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Logits of a tile, and of it those of a lane: 128 bytes a lane.
template <typename T>
constexpr int tile_each() { return 128 / static_cast<int>(sizeof(T)); }

// Sums over logits relative to m, in powers of 2: s = sum 2^u, w = sum 2^u u, u = (z - m) log2 e.
struct Part {
    float m, s, w;
};

// (z - m) log2 e. A logit below every finite one, or so far below the maximum that its weight is 0,
// must not multiply that 0 by an infinity; a NaN passes (v_maximum3_f32).
__device__ __forceinline__ float relative(float z, float m) {
    return __builtin_elementwise_maximum((z - m) * kLog2e, -1000.0f);
}

__device__ __forceinline__ void add_logit(Part &p, float z) {
    const float u = relative(z, p.m);
    const float e = __builtin_amdgcn_exp2f(u);
    p.s += e;
    p.w = fmaf(e, u, p.w);
}

// As add_logit for every one of a lane's logits, in one fused operation from z to the exponent: with
// c = m log2 e rounded and r what the rounding left, fma(z, log2 e, -c) is u + r. r, up to 2^-25 of c,
// has to stay small beside u: below 2^-8 up to the bound taken here, which fp16's lowest value is
// inside of. Beyond it the difference is taken first.
template <int EACH, class Logit>
__device__ __forceinline__ void add_logits(Part &p, const Logit &logit) {
    if (fabsf(p.m) <= 65536.0f) {
        const float c = p.m * kLog2e;
        const float r = fmaf(p.m, kLog2e, -c);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const float u = __builtin_elementwise_maximum(fmaf(logit(i), kLog2e, -c), -1000.0f);
            const float e = __builtin_amdgcn_exp2f(u);
            p.s += e;
            p.w = fmaf(e, u, p.w);
        }
        const float back = __builtin_amdgcn_exp2f(-r);
        p.w = back * fmaf(-r, p.s, p.w);
        p.s *= back;
    } else {
#pragma unroll
        for (int i = 0; i < EACH; ++i) add_logit(p, logit(i));
    }
}

// The part's sums relative to another m.
__device__ __forceinline__ Part moved(const Part &p, float m) {
    const float u = relative(p.m, m);
    const float e = __builtin_amdgcn_exp2f(u);
    return {m, p.s * e, e * fmaf(u, p.s, p.w)};
}

// Maximum and sum over groups of lanes, 8 to 64; both lanes of a pair combine the same two numbers.
template <int CONTROL, class V>
__device__ __forceinline__ V lane_pair(V v) {
    static_assert(sizeof(V) == 4, "a register");
    return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CONTROL, 0xF, 0xF, true));
}

template <int GROUP, class V, class Op>
__device__ __forceinline__ V over_lanes(V v, Op op) {
    v = op(v, lane_pair<0xB1>(v));   // quad_perm 1,0,3,2
    v = op(v, lane_pair<0x4E>(v));   // quad_perm 2,3,0,1
    v = op(v, lane_pair<0x141>(v));  // row_half_mirror: the other quad of eight
    if constexpr (GROUP > 8) v = op(v, lane_pair<0x140>(v));  // row_mirror: the other eight of sixteen
    if constexpr (GROUP > 16) v = op(v, __shfl_xor(v, 16));
    if constexpr (GROUP > 32) v = op(v, __shfl_xor(v, 32));
    return v;
}

template <int GROUP>
__device__ __forceinline__ float most_over_lanes(float v) {
    return over_lanes<GROUP>(v, [](float a, float b) { return fmaxf(a, b); });
}

template <int GROUP>
__device__ __forceinline__ float sum_over_lanes(float v) {
    return over_lanes<GROUP>(v, [](float a, float b) { return a + b; });
}

// Four waves' parts as one; every thread of the workgroup gets it. Ends with the sums read.
__device__ __forceinline__ Part join_waves(const Part &p, Part (&parts)[kWaves]) {
    if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = p;
    __syncthreads();
    const float m = fmaxf(fmaxf(parts[0].m, parts[1].m), fmaxf(parts[2].m, parts[3].m));
    Part all = {m, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const Part one = moved(parts[i], m);
        all.s += one.s;
        all.w += one.w;
    }
    return all;
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

// The largest key of the workgroup. Called in turns: the barriers keep one turn's keys from the next's.
__device__ __forceinline__ Key most_of_waves(Key k, Key (&round)[kWaves]) {
    k = most_of_lanes<64>(k);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) round[threadIdx.x >> 6] = k;
    __syncthreads();
    k = round[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) k = round[w] > k ? round[w] : k;
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
    if (lane == 0) a.entropy[row] = empty ? 0.0f : log_s - p.w / p.s * kLn2;
    for (int r = lane; r < a.top; r += lanes) write_top(a, row, r, keys, p.m, log_s, empty);
}

// ---- small vocabularies ------------------------------------------------------------------

template <typename T, int GROUP, int EACH>
__global__ __launch_bounds__(kThreads) void small_kernel(LogprobArgs a) {
    __shared__ Key tops[kThreads / GROUP][kMostTop];
    const int lane = threadIdx.x % GROUP;
    const int group = threadIdx.x / GROUP;
    const long long row = static_cast<long long>(workgroup_number()) * (kThreads / GROUP) + group;
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
    p.m = most_over_lanes<GROUP>(p.m);
    add_logits<EACH>(p, [&](int i) { return z[i]; });
    p.s = sum_over_lanes<GROUP>(p.s);
    p.w = sum_over_lanes<GROUP>(p.w);
    if (a.top > 0) {
        unsigned left[EACH];  // ordered bits, 0 for a masked token, one past the row or one listed
#pragma unroll
        for (int i = 0; i < EACH; ++i) left[i] = masked(z[i]) ? 0 : ordered(z[i]);
        for (int r = 0; r < a.top; ++r) {
            unsigned best = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i) best = left[i] > best ? left[i] : best;
            best = over_lanes<GROUP>(best, [](unsigned u, unsigned v) { return u > v ? u : v; });
            int token = 0x7FFFFFFF;
#pragma unroll
            for (int i = EACH - 1; i >= 0; --i) token = left[i] == best ? i * GROUP + lane : token;
            token = over_lanes<GROUP>(token, [](int u, int v) { return u < v ? u : v; });
#pragma unroll
            for (int i = 0; i < EACH; ++i) left[i] = i * GROUP + lane == token ? 0 : left[i];
            if (lane == 0) tops[group][r] = best == 0 ? 0 : (static_cast<Key>(best) << 32) | static_cast<unsigned>(~token);
        }
    }
    __syncthreads();
    if (live) finish_row<T>(a, row, p, lane, GROUP, [&](int r) { return tops[group][r]; });
}

// ---- tiles -------------------------------------------------------------------------------

__host__ __device__ inline size_t part_words(int top) { return 2 + static_cast<size_t>(top); }  // 64-bit words of a tile

// Waves a SIMD that the registers are fitted to: 7, for 72 of them (74 cost 4 % of 512 x 100003 bfloat16).
// Whole bfloat16 rows would spill there: 2048 of 16000 tokens 29.6 us, 22.2 with as many as they take.
template <typename T, bool WHOLE>
constexpr int tile_waves() { return WHOLE && std::is_same<T, __bf16>::value ? 4 : 7; }

template <typename T, bool WHOLE>
__global__ __launch_bounds__(kThreads, (tile_waves<T, WHOLE>())) void tile_kernel(LogprobArgs a, int tiles) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    constexpr int kEach = tile_each<T>();
    constexpr int kVectors = kEach / V;
    __shared__ Part parts[kWaves];
    __shared__ unsigned reach[kWaves];
    __shared__ Key list[kList];
    __shared__ Key top[kMostTop];
    __shared__ Key round[kWaves];
    __shared__ int listed;

    const int tid = threadIdx.x;
    const int wave = tid >> 6;
    const long long row = __builtin_amdgcn_readfirstlane(static_cast<int>(workgroup_number() / static_cast<unsigned>(tiles)));
    const int tile = __builtin_amdgcn_readfirstlane(static_cast<int>(workgroup_number() % static_cast<unsigned>(tiles)));
    if (row >= a.rows) return;
    const T *x = static_cast<const T *>(a.logits) + row * a.stride;
    // vector n of the row holds tokens n V - skew .. n V - skew + V - 1, 16-byte aligned
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int first = (tile * kVectors * kThreads + tid) * V - skew;  // of this lane's first vector
    const T masked_out = static_cast<T>(-__builtin_huge_valf());
    typedef unsigned int Raw __attribute__((ext_vector_type(4)));
    Raw raw[kVectors];
    if (tile * kEach * kThreads >= skew && (tile + 1) * kEach * kThreads - skew <= a.vocabulary) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) raw[i] = *reinterpret_cast<const Raw *>(x + first + i * kThreads * V);
    } else {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int t = first + i * kThreads * V;
            if (t >= 0 && t + V <= a.vocabulary) {
                raw[i] = *reinterpret_cast<const Raw *>(x + t);
            } else {
                Vec<T, V> v;
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = t + e >= 0 && t + e < a.vocabulary ? x[t + e] : masked_out;
                raw[i] = __builtin_bit_cast(Raw, v);
            }
        }
    }
    auto logit = [&](int i) { return static_cast<float>(__builtin_bit_cast(Vec<T, V>, raw[i / V])[i % V]); };
    // The logits stay as they came, 32 registers; widened ones are not kept from one pass over them to the
    // next (the compiler would).
    auto forget_widened = [&] {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < kVectors; ++i) asm volatile("" : "+v"(raw[i]));
        }
    };
    auto token = [&](int i) { return first + i / V * kThreads * V + i % V; };
    if (tid == 0) listed = 0;
    if (tid < kMostTop) top[tid] = 0;

    float lane_most = kLowest, vector_most[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        vector_most[i] = kLowest;
#pragma unroll
        for (int e = 0; e < V; ++e) vector_most[i] = fmaxf(vector_most[i], logit(i * V + e));
        lane_most = fmaxf(lane_most, vector_most[i]);
    }
    Part p = {most_over_lanes<64>(lane_most), 0.0f, 0.0f};
    forget_widened();
    add_logits<kEach>(p, logit);
    forget_widened();
    const bool lane_nan = p.s != p.s;  // or infinite: then its maximum is
    p.s = sum_over_lanes<64>(p.s);
    p.w = sum_over_lanes<64>(p.w);
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
    p = join_waves(p, parts);
    if (a.top > 0) {
        unsigned bound = reach[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) bound = reach[w] > bound ? reach[w] : bound;
        const float least = from_ordered(bound);  // at least kLowest, as every lane's maximum is: nothing masked reaches it
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            if (!__any(lane_nan || vector_most[i] >= least)) continue;
#pragma unroll
            for (int e = i * V; e < (i + 1) * V; ++e) {
                const bool found = !(logit(e) < least);  // a NaN too
                if (found) {
                    const int at = atomicAdd(&listed, 1);
                    if (at < kList) list[at] = key_of(logit(e), token(e));
                }
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
                // from the caches again: 64 keys a lane at once would not fit the registers
                Key best = 0;
#pragma unroll 1
                for (int i = 0; i < kVectors; ++i) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int t = first + i * kThreads * V + e;
                        const Key k = t >= 0 && t < a.vocabulary ? key_of(static_cast<float>(x[t]), t) : 0;
                        best = k < last && k > best ? k : best;
                    }
                }
                last = most_of_waves(best, round);
                if (tid == 0) top[r] = last;
            }
            __syncthreads();
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

// A workgroup joins the tiles of a row: thread t takes tile t's part; the tiles' top keys, all
// different, are ranked by counting, or, where there are many, taken by `top` rounds of a maximum.
template <typename T>
__global__ __launch_bounds__(kThreads) void join_kernel(LogprobArgs a, int tiles) {
    constexpr int kRanked = 512;
    __shared__ Part parts[kWaves];
    __shared__ Key keys[kMostTiles * kMostTop];
    __shared__ Key top[kMostTop];
    __shared__ Key round[kWaves];
    static_assert(kMostTiles <= kThreads, "a tile a thread");
    const int tid = threadIdx.x;
    const long long row = workgroup_number();
    if (row >= a.rows) return;
    const int words = static_cast<int>(part_words(a.top));
    const Key *in = static_cast<const Key *>(a.scratch) + static_cast<size_t>(row) * tiles * words;
    const int n = tiles * a.top;
    for (int i = tid; i < n; i += kThreads) keys[i] = in[i / a.top * words + 2 + i % a.top];
    Part p = {kLowest, 0.0f, 0.0f};
    if (tid < tiles) {
        const Key one = in[tid * words], two = in[tid * words + 1];
        p = {__uint_as_float(static_cast<unsigned>(one)), __uint_as_float(static_cast<unsigned>(one >> 32)),
             __uint_as_float(static_cast<unsigned>(two))};
    }
    if (tid < kMostTop) top[tid] = 0;
    p = moved(p, most_over_lanes<64>(p.m));
    p.s = sum_over_lanes<64>(p.s);
    p.w = sum_over_lanes<64>(p.w);
    p = join_waves(p, parts);
    if (n <= kRanked) {
        for (int i = tid; i < n; i += kThreads) {
            const Key mine = keys[i];
            if (mine == 0) continue;
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += keys[j] > mine ? 1 : 0;
            if (rank < a.top) top[rank] = mine;
        }
    } else {
        Key last = ~static_cast<Key>(0);
        for (int r = 0; r < a.top; ++r) {
            Key best = 0;
            for (int i = tid; i < n; i += kThreads) best = keys[i] < last && keys[i] > best ? keys[i] : best;
            last = most_of_waves(best, round);
            if (tid == 0) top[r] = last;
        }
    }
    __syncthreads();
    finish_row<T>(a, row, p, tid, kThreads, [&](int r) { return top[r]; });
}

// Tiles of a row, whatever its alignment: a vector's first tokens may belong to the row before.
template <typename T>
int tiles_of(int vocabulary) {
    constexpr int kTile = kThreads * tile_each<T>(), kSkew = 16 / static_cast<int>(sizeof(T)) - 1;
    return (vocabulary + kSkew + kTile - 1) / kTile;
}

template <typename T, int GROUP, int EACH>
hipError_t run_small(const LogprobArgs &a, hipStream_t stream) {
    constexpr int kRows = kThreads / GROUP;
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.rows) + kRows - 1) / kRows);
    return launch(small_kernel<T, GROUP, EACH>, blocks, kThreads, stream, a);
}

// A row in a wave needs no barrier and leaves few lanes idle, but its rounds go over all of a lane's
// logits: kSmall logits, twice as many if few alternatives are asked for. A wave against a tile a row,
// us, with 0, 5 and 32 alternatives: 4096 rows of 1000 bfloat16 5.8/26, 10.5/32.5 and 29.8/38.5; 2048 rows
// of 2048 7.6/15.2, 12.2/19.0 and 31.6/24.5; float32 4.6/9.0, 9.8/12.5 and 29.1/18.3; 1024 rows of 4096
// bfloat16 10.9/8.7, 18.7/11.9 and 49/16. A group as wide as the row needs: with 4 and 16 logits a lane
// 16384 rows of 256 float32 take 12.4 and 23.1 us; 131072 rows of 32 take 16 us on 16 lanes, 36 on 32.
bool is_small(int vocabulary, int top) { return vocabulary <= kSmall || (vocabulary <= 2 * kSmall && top <= 8); }

template <typename T>
hipError_t run(const LogprobArgs &a, hipStream_t stream) {
    if (a.vocabulary <= 8) return run_small<T, 8, 1>(a, stream);
    if (a.vocabulary <= 32) return run_small<T, 16, 2>(a, stream);
    if (a.vocabulary <= 128) return run_small<T, 32, 4>(a, stream);
    if (a.vocabulary <= 256) return run_small<T, 64, 4>(a, stream);
    if (a.vocabulary <= 512) return run_small<T, 64, 8>(a, stream);
    if (a.vocabulary <= kSmall) return run_small<T, 64, kSmall / 64>(a, stream);
    if (is_small(a.vocabulary, a.top)) return run_small<T, 64, kSmall / 32>(a, stream);
    const int tiles = tiles_of<T>(a.vocabulary);
    const unsigned long long blocks = static_cast<unsigned long long>(a.rows) * static_cast<unsigned>(tiles);
    if (tiles == 1) return launch(tile_kernel<T, true>, blocks, kThreads, stream, a, tiles);
    const hipError_t e = launch(tile_kernel<T, false>, blocks, kThreads, stream, a, tiles);
    if (e != hipSuccess) return e;
    return launch(join_kernel<T>, static_cast<unsigned long long>(a.rows), kThreads, stream, a, tiles);
}

}  // namespace

size_t logprob_scratch_bytes(int rows, int vocabulary, int top, Elem type) {
    const int tiles = type == Elem::f32 ? tiles_of<float>(vocabulary) : tiles_of<__bf16>(vocabulary);
    if (is_small(vocabulary, top) || tiles == 1) return 0;
    return static_cast<size_t>(rows) * tiles * part_words(top) * sizeof(Key);
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
