// Device helpers of cross attention: who reads which memory, and the two products' operands.
#pragma once

#include "tile_device.h"

namespace bl {

typedef float F16x __attribute__((ext_vector_type(16)));  // a 32 x 32 accumulator's share of a lane
typedef unsigned int U4 __attribute__((ext_vector_type(4)));

// What one workgroup does: `count` packed rows from `first` on (row i * per + h is head g * per + h of row i of the
// sequence) of one group of heads, over the frames begin .. end - 1 of its memory.
struct Work {
    long long row;      // the sequence's first row
    long long first;    // packed rows of the sequence
    int count;          // 0: nothing to do
    int group;
    int split;
    long long memory;   // the memory's first row
    int begin, end;     // frames
};

// Tiles of `size` packed rows never cross a sequence; they are numbered like runs of rows (see sequence_of_run).
__device__ __forceinline__ long long tile_base(const AttentionArgs &a, int j, int size) {
    return static_cast<long long>(clamp_row(a.seq.starts[j], a.seq.rows)) * a.per / size + j;
}

__device__ __forceinline__ Work work_of(const AttentionArgs &a, int size, int frames) {
    Work w;
    w.count = 0;
    unsigned number = workgroup_number();
    w.group = static_cast<int>(number % a.groups);
    number /= a.groups;
    w.split = static_cast<int>(number % a.splits);
    const long long tile = number / a.splits;
    int j;
    long long left;  // packed rows of the sequence from the tile's first on
    if (a.seq.starts == nullptr) {
        const int each = (a.per + size - 1) / size;
        if (tile / each >= a.seq.sequences) return w;
        j = static_cast<int>(tile / each);
        w.row = j;
        w.first = tile % each * size;
        left = a.per - w.first;
    } else {
        j = last_sequence_wave(a.seq, [&](int i) { return tile_base(a, i, size) <= tile; });
        const Span span = span_of(a.seq, j);
        const long long at = tile - tile_base(a, j, size);
        if (at < 0) return w;  // before the first sequence
        w.row = span.first;
        w.first = at * size;
        left = static_cast<long long>(span.length) * a.per - w.first;
    }
    const int place = place_of(a.seq, j);
    if (left <= 0 || place < 0) return w;
    w.count = left < size ? static_cast<int>(left) : size;
    const int from = clamp_row(a.memory_starts[place], a.memory_rows), to = clamp_row(a.memory_starts[place + 1], a.memory_rows);
    int held = to > from ? to - from : 0;
    if (a.memory_lengths != nullptr) {
        const int length = a.memory_lengths[place];
        held = length < held ? (length > 0 ? length : 0) : held;
    }
    w.memory = from;
    const long long tiles = (static_cast<long long>(held) + frames - 1) / frames;
    w.begin = static_cast<int>(tiles * w.split / a.splits) * frames;
    const long long end = tiles * (w.split + 1) / a.splits * frames;
    w.end = end < held ? static_cast<int>(end) : held;
    return w;
}

// Splits' parts: per split, row and head the quotients of its frames alone, then per split, row and head the
// score that weights are measured from (without the scale) and the sum of weights.
__device__ __forceinline__ float *part_values(const AttentionArgs &a, int split, long long row, int head) {
    return a.scratch + ((static_cast<size_t>(split) * a.seq.rows + row) * a.heads + head) * a.padded;
}

__device__ __forceinline__ float *part_sums(const AttentionArgs &a, int split, long long row, int head) {
    float *const from = a.scratch + static_cast<size_t>(a.splits) * a.seq.rows * a.heads * a.padded;
    return from + ((static_cast<size_t>(split) * a.seq.rows + row) * a.heads + head) * 2;
}

}  // namespace bl
