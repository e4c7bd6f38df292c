// Internal declarations of the causal sequence operators (convolution, state space scan, norm,
// token log probabilities): what the host side hands to the kernels. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace bl {

enum class Elem { f32, bf16, f16 };

// Packed sequences and the cache places that go with them; see include/bilstm.h. In the
// single-token form, without starts, row i is sequence i.
struct SequenceArgs {
    const int *starts = nullptr;
    const int *slots = nullptr;
    const unsigned char *fresh = nullptr;
    int sequences = 0;
    int places = 0;
    int rows = 0;
};

struct ConvArgs {
    const void *x = nullptr;
    const void *weight = nullptr;
    const void *bias = nullptr;
    void *state = nullptr;
    void *y = nullptr;
    size_t x_stride = 0, y_stride = 0;
    int channels = 0;
    int taps = 0;
    bool silu = false;
    SequenceArgs seq;
};

hipError_t launch_conv(const ConvArgs &args, Elem type, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs &args, Elem type, hipStream_t stream);

struct ScanArgs {
    const void *x = nullptr, *dt = nullptr, *b = nullptr, *c = nullptr, *z = nullptr;
    const float *a = nullptr, *d = nullptr, *dt_bias = nullptr;
    float *state = nullptr;
    void *y = nullptr;
    size_t x_stride = 0, dt_stride = 0, b_stride = 0, c_stride = 0, z_stride = 0, y_stride = 0;
    int heads = 0, width = 0, groups = 0, states = 0;
    bool softplus = false;
    SequenceArgs seq;
    void *scratch = nullptr;
};

size_t scan_scratch_bytes(const ScanArgs &args);
hipError_t launch_scan(const ScanArgs &args, Elem type, hipStream_t stream);
hipError_t launch_scan_step(const ScanArgs &args, Elem type, hipStream_t stream);

enum class Eight { none, e4m3, int8 };

struct NormArgs {
    const void *x = nullptr, *residual = nullptr, *weight = nullptr;
    void *residual_out = nullptr, *y = nullptr;
    unsigned char *q = nullptr;
    float *scales = nullptr;
    size_t x_stride = 0, residual_stride = 0, residual_out_stride = 0, y_stride = 0, q_stride = 0;
    int rows = 0;
    int width = 0;
    double inverse_width = 0.0;
    float eps = 0.0f;
};

hipError_t launch_add_rms_norm(const NormArgs &args, Elem type, Eight eight, hipStream_t stream);

struct LogprobArgs {
    const void *logits = nullptr;
    size_t stride = 0;
    const long long *tokens = nullptr;
    float *logprobs = nullptr;
    float *entropy = nullptr;
    long long *top_tokens = nullptr;
    float *top_logprobs = nullptr;
    void *scratch = nullptr;
    int rows = 0;
    int vocabulary = 0;
    int given = 0;
    int top = 0;
};

constexpr int kMostTop = 32;
size_t logprob_scratch_bytes(int rows, int vocabulary, int top, Elem type);
hipError_t launch_token_logprobs(const LogprobArgs &args, Elem type, hipStream_t stream);

// Sequences of rows (or, with `step`, single rows) that read memories: places are the memories.
struct AttentionArgs {
    const void *q = nullptr, *k = nullptr, *v = nullptr;
    const int *memory_starts = nullptr;
    const int *memory_lengths = nullptr;
    const unsigned char *mask = nullptr;
    void *y = nullptr;
    float *scratch = nullptr;
    size_t q_stride = 0, k_stride = 0, v_stride = 0, y_stride = 0;
    int heads = 0, groups = 0, width = 0;
    int per = 0;  // heads that share keys and values
    int memory_rows = 0;
    float scale = 0.0f;
    bool step = false;
    SequenceArgs seq;
    int splits = 0, padded = 0;  // the launch's own
};

size_t attention_scratch_bytes(const AttentionArgs &args);
hipError_t launch_attention(const AttentionArgs &args, Elem type, hipStream_t stream);

struct LinearArgs {
    const void *x = nullptr, *weight = nullptr, *bias = nullptr, *residual = nullptr;
    const float *x_scales = nullptr, *weight_scales = nullptr;
    void *y = nullptr;
    float *scratch = nullptr;
    size_t x_stride = 0, weight_stride = 0, residual_stride = 0, y_stride = 0;
    int rows = 0, in = 0, out = 0;
    int activation = 0;
    float slope = 0.0f;
    int steps = 0, splits = 0, tiles_m = 0, tiles_n = 0, whole = 0;  // the launch's own
};

size_t linear_scratch_bytes(const LinearArgs &args, Elem type, Eight eight);
hipError_t launch_linear(const LinearArgs &args, Elem type, Eight eight, hipStream_t stream);

}  // namespace bl
