// C ABI of the causal sequence operators: checks of arguments, then one launcher call. These
// entry points keep nothing between calls and allocate nothing.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "../../include/bilstm.h"
#include "bilstm_host.h"
#include "sequence_internal.h"

using namespace bl;

namespace {

constexpr uint64_t kMostRows = 0x7FFFFFFFull;
constexpr uint32_t kMostSequences = 1u << 30;

// Byte range of a view, for overlap checks; strided views repeat `width` bytes every `stride`.
struct Bytes {
    uintptr_t first = 0;
    uint64_t rows = 0, width = 0, stride = 0;
    bool empty() const { return rows == 0 || width == 0 || first == 0; }
    uintptr_t end() const { return first + (rows - 1) * stride + width; }
};

Bytes bytes_of(const bilstm_rows &r, uint64_t rows, uint64_t width, uint64_t size) {
    return {reinterpret_cast<uintptr_t>(r.data), rows, width * size, r.stride * size};
}

Bytes bytes_of(const bilstm_buffer &b, uint64_t size) {
    return {reinterpret_cast<uintptr_t>(b.data), b.data != nullptr ? 1ull : 0ull, b.len * size, b.len * size};
}

// Whether two views share a byte. Views of one wide buffer with the same stride may interleave:
// they are apart if their columns are.
bool overlap(const Bytes &a, const Bytes &b) {
    if (a.empty() || b.empty()) return false;
    if (a.end() <= b.first || b.end() <= a.first) return false;
    if (a.stride == b.stride && a.rows > 1 && b.rows > 1) {
        const uint64_t off = a.first <= b.first ? (b.first - a.first) % a.stride
                                                : (a.stride - (a.first - b.first) % a.stride) % a.stride;
        return off < a.width || off + b.width > a.stride;
    }
    return true;
}

bool same_view(const bilstm_rows &a, const bilstm_rows &b, uint64_t rows) {
    return a.data == b.data && (rows <= 1 || a.stride == b.stride);
}

uint64_t size_of(int32_t type) { return type == BILSTM_FLOAT32 ? 4 : 2; }
Elem elem_of(int32_t type) {
    return type == BILSTM_FLOAT32 ? Elem::f32 : (type == BILSTM_BFLOAT16 ? Elem::bf16 : Elem::f16);
}

bilstm_status check_type(const char *call, int32_t type) {
    if (type < BILSTM_FLOAT32 || type > BILSTM_FLOAT16) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: unknown element type %d", call, type);
    }
    return BILSTM_OK;
}

bilstm_status check_pointer(const char *call, const char *name, const void *p, uint64_t align) {
    if (p == nullptr) return fail(BILSTM_INVALID_ARGUMENT, "%s: %s is NULL", call, name);
    if (reinterpret_cast<uintptr_t>(p) % align != 0) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: %s must be %llu-byte aligned", call, name,
                    static_cast<unsigned long long>(align));
    }
    return BILSTM_OK;
}

bilstm_status check_rows(const char *call, const char *name, const bilstm_rows &r, uint64_t rows, uint64_t width,
                         uint64_t size) {
    bilstm_status st = check_pointer(call, name, r.data, size);
    if (st != BILSTM_OK) return st;
    if (r.stride < width && rows > 1) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: %s has a row stride of %llu, less than its width %llu", call, name,
                    static_cast<unsigned long long>(r.stride), static_cast<unsigned long long>(width));
    }
    uint64_t need = 0, bytes = 0;
    if (__builtin_mul_overflow(rows - 1, r.stride, &need) || __builtin_add_overflow(need, width, &need) ||
        __builtin_mul_overflow(need, size, &bytes) || bytes > (1ull << 56) || r.stride > (1ull << 56)) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: %s does not fit the address space", call, name);
    }
    if (r.len < need) {
        return fail(BILSTM_BUFFER_LENGTH, "%s: %s: expected at least %llu elements, got %llu", call, name,
                    static_cast<unsigned long long>(need), static_cast<unsigned long long>(r.len));
    }
    return BILSTM_OK;
}

// `expected` elements exactly; optional buffers may be NULL.
bilstm_status check_buffer(const char *call, const char *name, const bilstm_buffer &b, uint64_t expected, uint64_t align,
                           bool optional) {
    if (b.data == nullptr && optional) return BILSTM_OK;
    bilstm_status st = check_pointer(call, name, b.data, align);
    if (st != BILSTM_OK) return st;
    if (b.len != expected) {
        return fail(BILSTM_BUFFER_LENGTH, "%s: %s: expected %llu elements, got %llu", call, name,
                    static_cast<unsigned long long>(expected), static_cast<unsigned long long>(b.len));
    }
    return BILSTM_OK;
}

bilstm_status check_apart(const char *call, const char *out_name, const Bytes &out, const char *in_name, const Bytes &in) {
    if (overlap(out, in)) return fail(BILSTM_INVALID_ARGUMENT, "%s: %s and %s overlap", call, out_name, in_name);
    return BILSTM_OK;
}

#define BL_CHECK(expr)                          \
    do {                                        \
        const bilstm_status st_ = (expr);       \
        if (st_ != BILSTM_OK) return st_;       \
    } while (0)

// Makes `device` current for a launch and the caller's device current again afterwards.
class DeviceScope {
  public:
    explicit DeviceScope(int device) : device_(device) {}
    bilstm_status enter(const char *call) {
        constexpr int kKnown = 64;
        static std::atomic<int> known[kKnown];  // 0 not looked at yet, 1 gfx950
        hipError_t e = hipSuccess;
        if (device_ < 0 || device_ >= kKnown || known[device_].load(std::memory_order_relaxed) == 0) {
            int count = 0;
            e = hipGetDeviceCount(&count);
            if (e != hipSuccess || count == 0) {
                return fail(BILSTM_UNSUPPORTED, "%s: no HIP device (%s)", call, hipGetErrorString(e));
            }
            if (device_ < 0 || device_ >= count) {
                return fail(BILSTM_INVALID_ARGUMENT, "%s: device %d out of range (%d devices)", call, device_, count);
            }
            hipDeviceProp_t prop;
            e = hipGetDeviceProperties(&prop, device_);
            if (e != hipSuccess) return fail(BILSTM_HIP_ERROR, "%s: device properties: %s", call, hipGetErrorString(e));
            if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) {
                return fail(BILSTM_UNSUPPORTED, "%s: device %d is not a gfx950 (MI355X) GPU", call, device_);
            }
            if (device_ < kKnown) known[device_].store(1, std::memory_order_relaxed);
        }
        e = hipGetDevice(&saved_);
        if (e == hipSuccess && saved_ != device_) {
            e = hipSetDevice(device_);
            switched_ = e == hipSuccess;
        }
        if (e != hipSuccess) return fail(BILSTM_HIP_ERROR, "%s: hipSetDevice: %s", call, hipGetErrorString(e));
        return BILSTM_OK;
    }
    ~DeviceScope() {
        if (switched_) (void)hipSetDevice(saved_);
    }
    DeviceScope(const DeviceScope &) = delete;
    DeviceScope &operator=(const DeviceScope &) = delete;

  private:
    int device_;
    int saved_ = 0;
    bool switched_ = false;
};

bilstm_status launched(const char *call, hipError_t e) {
    if (e == hipErrorInvalidConfiguration) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: more work than one launch's grid holds", call);
    }
    if (e != hipSuccess) return fail(BILSTM_HIP_ERROR, "%s: launch: %s", call, hipGetErrorString(e));
    return BILSTM_OK;
}

// The sequences of a call: numbers, starts, slots, fresh.
template <class Args>
bilstm_status check_sequences(const char *call, const Args &a, bool step, SequenceArgs *s) {
    if (a.rows > kMostRows) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: %llu rows exceed 32-bit row numbers", call,
                    static_cast<unsigned long long>(a.rows));
    }
    if (a.reserved != 0) return fail(BILSTM_INVALID_ARGUMENT, "%s: reserved must be 0", call);
    const uint64_t count = step ? a.rows : a.sequences;
    if (count > kMostSequences || a.places > kMostRows) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: too many sequences or places", call);
    }
    if (!step && count > 0) BL_CHECK(check_buffer(call, "starts", a.starts, count + 1, 4, false));
    if (count > 0) BL_CHECK(check_buffer(call, "slots", a.slots, count, 4, true));
    if (!step && count > 0) BL_CHECK(check_buffer(call, "fresh", a.fresh, count, 1, true));
    if (a.state.data == nullptr && (step || a.slots.data != nullptr || a.fresh.data != nullptr)) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: %s", call,
                    step ? "the single-token form needs a state" : "slots and fresh need a state");
    }
    if (a.state.data != nullptr && a.slots.data == nullptr && count > a.places) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: %llu sequences without slots, but only %u places", call,
                    static_cast<unsigned long long>(count), a.places);
    }
    s->starts = step ? nullptr : static_cast<const int *>(a.starts.data);
    s->slots = static_cast<const int *>(a.slots.data);
    s->fresh = step ? nullptr : static_cast<const unsigned char *>(a.fresh.data);
    s->sequences = static_cast<int>(count);
    s->places = static_cast<int>(a.places);
    s->rows = static_cast<int>(a.rows);
    return BILSTM_OK;
}

// ---- convolution -------------------------------------------------------------------------

bilstm_status conv(const char *call, const bilstm_conv_args *args, bool step, void *stream) {
    if (args == nullptr) return fail(BILSTM_INVALID_ARGUMENT, "%s: args is NULL", call);
    const bilstm_conv_args &a = *args;
    BL_CHECK(check_type(call, a.type));
    if (a.channels == 0 || a.channels > kMostRows) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: %u channels", call, a.channels);
    }
    if (a.taps < 2 || a.taps > 4) return fail(BILSTM_UNSUPPORTED, "%s: %u taps (2, 3 or 4 are built)", call, a.taps);
    ConvArgs k;
    BL_CHECK(check_sequences(call, a, step, &k.seq));
    if (a.rows == 0 || k.seq.sequences == 0) return BILSTM_OK;
    const uint64_t size = size_of(a.type);
    BL_CHECK(check_rows(call, "x", a.x, a.rows, a.channels, size));
    BL_CHECK(check_rows(call, "y", a.y, a.rows, a.channels, size));
    BL_CHECK(check_buffer(call, "weight", a.weight, static_cast<uint64_t>(a.channels) * a.taps, size, false));
    BL_CHECK(check_buffer(call, "bias", a.bias, a.channels, size, true));
    uint64_t state_len = 0;
    if (__builtin_mul_overflow(static_cast<uint64_t>(a.places), static_cast<uint64_t>(a.channels) * (a.taps - 1),
                               &state_len) || state_len > (1ull << 54)) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: state does not fit the address space", call);
    }
    BL_CHECK(check_buffer(call, "state", a.state, state_len, size, true));
    const Bytes x = bytes_of(a.x, a.rows, a.channels, size), y = bytes_of(a.y, a.rows, a.channels, size);
    const Bytes state = bytes_of(a.state, size);
    BL_CHECK(check_apart(call, "y", y, "x", x));
    BL_CHECK(check_apart(call, "y", y, "state", state));
    BL_CHECK(check_apart(call, "state", state, "x", x));
    const bilstm_buffer none = {nullptr, 0};
    const Bytes inputs[] = {bytes_of(a.weight, size), bytes_of(a.bias, size), bytes_of(step ? none : a.starts, 4),
                            bytes_of(a.slots, 4), bytes_of(step ? none : a.fresh, 1)};
    for (const Bytes &in : inputs) {
        BL_CHECK(check_apart(call, "y", y, "an input", in));
        BL_CHECK(check_apart(call, "state", state, "an input", in));
    }
    k.x = a.x.data;
    k.weight = a.weight.data;
    k.bias = a.bias.data;
    k.state = const_cast<void *>(a.state.data);
    k.y = const_cast<void *>(a.y.data);
    k.x_stride = a.x.stride;
    k.y_stride = a.y.stride;
    k.channels = static_cast<int>(a.channels);
    k.taps = static_cast<int>(a.taps);
    k.silu = a.silu != 0;
    DeviceScope scope(a.device);
    BL_CHECK(scope.enter(call));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return launched(call, step ? launch_conv_step(k, elem_of(a.type), s) : launch_conv(k, elem_of(a.type), s));
}

// ---- scan ----------------------------------------------------------------------------------

// The sizes of a scan, without its pointers.
bilstm_status scan_sizes(const char *call, const bilstm_scan_args *args, bool step, ScanArgs *k) {
    if (args == nullptr) return fail(BILSTM_INVALID_ARGUMENT, "%s: args is NULL", call);
    const bilstm_scan_args &a = *args;
    BL_CHECK(check_type(call, a.type));
    if (a.heads == 0 || a.groups == 0 || a.heads % a.groups != 0) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: %u heads in %u groups", call, a.heads, a.groups);
    }
    if (a.width != 32 && a.width != 64 && a.width != 128) {
        return fail(BILSTM_UNSUPPORTED, "%s: heads of %u channels (32, 64 and 128 are built)", call, a.width);
    }
    if (a.states != 16 && a.states != 32 && a.states != 64 && a.states != 128 && a.states != 256) {
        return fail(BILSTM_UNSUPPORTED, "%s: %u states (16, 32, 64, 128 and 256 are built)", call, a.states);
    }
    if (static_cast<uint64_t>(a.heads) * a.width * a.states > (1u << 30) || a.rows > kMostRows ||
        (!step && a.sequences > kMostSequences)) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: %llu rows of %u heads exceed the kernels' indexing", call,
                    static_cast<unsigned long long>(a.rows), a.heads);
    }
    k->heads = static_cast<int>(a.heads);
    k->width = static_cast<int>(a.width);
    k->groups = static_cast<int>(a.groups);
    k->states = static_cast<int>(a.states);
    k->seq.rows = static_cast<int>(a.rows);
    k->seq.sequences = static_cast<int>(step ? a.rows : a.sequences);
    return BILSTM_OK;
}

bilstm_status scan(const char *call, const bilstm_scan_args *args, bool step, void *stream) {
    ScanArgs k;
    BL_CHECK(scan_sizes(call, args, step, &k));
    const bilstm_scan_args &a = *args;
    BL_CHECK(check_sequences(call, a, step, &k.seq));
    if (a.rows == 0 || k.seq.sequences == 0) return BILSTM_OK;
    const uint64_t size = size_of(a.type);
    const uint64_t inner = static_cast<uint64_t>(a.heads) * a.width, shared = static_cast<uint64_t>(a.groups) * a.states;
    BL_CHECK(check_rows(call, "x", a.x, a.rows, inner, size));
    BL_CHECK(check_rows(call, "dt", a.dt, a.rows, a.heads, size));
    BL_CHECK(check_rows(call, "b", a.b, a.rows, shared, size));
    BL_CHECK(check_rows(call, "c", a.c, a.rows, shared, size));
    if (a.z.data != nullptr) BL_CHECK(check_rows(call, "z", a.z, a.rows, inner, size));
    BL_CHECK(check_rows(call, "y", a.y, a.rows, inner, size));
    BL_CHECK(check_buffer(call, "a", a.a, a.heads, 4, false));
    BL_CHECK(check_buffer(call, "d", a.d, a.heads, 4, true));
    BL_CHECK(check_buffer(call, "dt_bias", a.dt_bias, a.heads, 4, true));
    uint64_t state_len = 0;
    if (__builtin_mul_overflow(static_cast<uint64_t>(a.places), inner * a.states, &state_len) || state_len > (1ull << 54)) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: state does not fit the address space", call);
    }
    BL_CHECK(check_buffer(call, "state", a.state, state_len, 16, true));
    const uint64_t need = step ? 0 : scan_scratch_bytes(k);
    if (need > 0) {
        BL_CHECK(check_pointer(call, "scratch", a.scratch.data, 16));
        if (a.scratch.len < need) {
            return fail(BILSTM_BUFFER_LENGTH, "%s: scratch: expected at least %llu bytes, got %llu", call,
                        static_cast<unsigned long long>(need), static_cast<unsigned long long>(a.scratch.len));
        }
    }
    struct Region {
        const char *name;
        Bytes bytes;
    };
    const bilstm_rows no_rows = {nullptr, 0, 0};
    const bilstm_buffer none = {nullptr, 0};
    const Region ins[] = {{"x", bytes_of(a.x, a.rows, inner, size)},
                          {"dt", bytes_of(a.dt, a.rows, a.heads, size)},
                          {"b", bytes_of(a.b, a.rows, shared, size)},
                          {"c", bytes_of(a.c, a.rows, shared, size)},
                          {"z", bytes_of(a.z.data != nullptr ? a.z : no_rows, a.rows, inner, size)},
                          {"a", bytes_of(a.a, 4)},
                          {"d", bytes_of(a.d, 4)},
                          {"dt_bias", bytes_of(a.dt_bias, 4)},
                          {"starts", bytes_of(step ? none : a.starts, 4)},
                          {"slots", bytes_of(a.slots, 4)},
                          {"fresh", bytes_of(step ? none : a.fresh, 1)}};
    const Region outs[] = {{"y", bytes_of(a.y, a.rows, inner, size)},
                           {"state", bytes_of(a.state, 4)},
                           {"scratch", bytes_of(need > 0 ? a.scratch : none, 1)}};
    for (const Region &o : outs) {
        for (const Region &in : ins) BL_CHECK(check_apart(call, o.name, o.bytes, in.name, in.bytes));
        for (const Region &other : outs) {
            if (&other != &o) BL_CHECK(check_apart(call, o.name, o.bytes, other.name, other.bytes));
        }
    }
    k.x = a.x.data;
    k.dt = a.dt.data;
    k.b = a.b.data;
    k.c = a.c.data;
    k.z = a.z.data;
    k.a = static_cast<const float *>(a.a.data);
    k.d = static_cast<const float *>(a.d.data);
    k.dt_bias = static_cast<const float *>(a.dt_bias.data);
    k.state = static_cast<float *>(const_cast<void *>(a.state.data));
    k.y = const_cast<void *>(a.y.data);
    k.x_stride = a.x.stride;
    k.dt_stride = a.dt.stride;
    k.b_stride = a.b.stride;
    k.c_stride = a.c.stride;
    k.z_stride = a.z.data != nullptr ? a.z.stride : 0;
    k.y_stride = a.y.stride;
    k.softplus = a.softplus != 0;
    k.scratch = const_cast<void *>(a.scratch.data);
    DeviceScope scope(a.device);
    BL_CHECK(scope.enter(call));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return launched(call, step ? launch_scan_step(k, elem_of(a.type), s) : launch_scan(k, elem_of(a.type), s));
}

// ---- norm ----------------------------------------------------------------------------------

bilstm_status norm(const char *call, const bilstm_norm_args *args, void *stream) {
    if (args == nullptr) return fail(BILSTM_INVALID_ARGUMENT, "%s: args is NULL", call);
    const bilstm_norm_args &a = *args;
    BL_CHECK(check_type(call, a.type));
    if (a.reserved != 0) return fail(BILSTM_INVALID_ARGUMENT, "%s: reserved must be 0", call);
    if (a.eight < BILSTM_EIGHT_NONE || a.eight > BILSTM_EIGHT_INT8) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: unknown 8-bit type %d", call, a.eight);
    }
    if (a.width == 0) return fail(BILSTM_INVALID_ARGUMENT, "%s: width is 0", call);
    if (!(a.eps >= 0.0f) || a.eps > 3.0e38f) return fail(BILSTM_INVALID_ARGUMENT, "%s: eps is not a number >= 0", call);
    if (a.rows > kMostRows || a.width > (1u << 30)) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: %llu rows of %u exceed the kernel's indexing", call,
                    static_cast<unsigned long long>(a.rows), a.width);
    }
    const bool eight = a.eight != BILSTM_EIGHT_NONE;
    if (!eight && (a.q.data != nullptr || a.scales.data != nullptr)) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: q and scales need an 8-bit type", call);
    }
    if (!eight && a.y.data == nullptr && a.rows > 0) return fail(BILSTM_INVALID_ARGUMENT, "%s: y is NULL", call);
    if (a.rows == 0) return BILSTM_OK;
    const uint64_t size = size_of(a.type);
    BL_CHECK(check_rows(call, "x", a.x, a.rows, a.width, size));
    if (a.residual.data != nullptr) BL_CHECK(check_rows(call, "residual", a.residual, a.rows, a.width, size));
    BL_CHECK(check_buffer(call, "weight", a.weight, a.width, size, false));
    if (a.residual_out.data != nullptr) BL_CHECK(check_rows(call, "residual_out", a.residual_out, a.rows, a.width, size));
    if (a.y.data != nullptr) BL_CHECK(check_rows(call, "y", a.y, a.rows, a.width, size));
    if (eight) {
        BL_CHECK(check_rows(call, "q", a.q, a.rows, a.width, 1));
        BL_CHECK(check_buffer(call, "scales", a.scales, a.rows, 4, false));
    }
    struct Out {
        const char *name;
        const bilstm_rows *view;  // may be an input itself; nullptr: may not
        Bytes bytes;
    };
    const Out outs[] = {{"residual_out", &a.residual_out, bytes_of(a.residual_out, a.rows, a.width, size)},
                        {"y", &a.y, bytes_of(a.y, a.rows, a.width, size)},
                        {"q", nullptr, bytes_of(a.q, a.rows, a.width, 1)},
                        {"scales", nullptr, bytes_of(a.scales, 4)}};
    for (const Out &o : outs) {
        BL_CHECK(check_apart(call, o.name, o.bytes, "weight", bytes_of(a.weight, size)));
        for (const bilstm_rows *in : {&a.x, &a.residual}) {
            if (o.view != nullptr && same_view(*o.view, *in, a.rows)) continue;
            BL_CHECK(check_apart(call, o.name, o.bytes, in == &a.x ? "x" : "residual", bytes_of(*in, a.rows, a.width, size)));
        }
        for (const Out &other : outs) {
            if (&other != &o) BL_CHECK(check_apart(call, o.name, o.bytes, other.name, other.bytes));
        }
    }
    NormArgs k;
    k.x = a.x.data;
    k.residual = a.residual.data;
    k.weight = a.weight.data;
    k.residual_out = const_cast<void *>(a.residual_out.data);
    k.y = const_cast<void *>(a.y.data);
    k.q = static_cast<unsigned char *>(const_cast<void *>(a.q.data));
    k.scales = static_cast<float *>(const_cast<void *>(a.scales.data));
    k.x_stride = a.x.stride;
    k.residual_stride = a.residual.data != nullptr ? a.residual.stride : 0;
    k.residual_out_stride = a.residual_out.data != nullptr ? a.residual_out.stride : 0;
    k.y_stride = a.y.data != nullptr ? a.y.stride : 0;
    k.q_stride = eight ? a.q.stride : 0;
    k.rows = static_cast<int>(a.rows);
    k.width = static_cast<int>(a.width);
    k.inverse_width = 1.0 / a.width;
    k.eps = a.eps;
    DeviceScope scope(a.device);
    BL_CHECK(scope.enter(call));
    return launched(call, launch_add_rms_norm(k, elem_of(a.type), static_cast<Eight>(a.eight),
                                              static_cast<hipStream_t>(stream)));
}

// ---- token log probabilities ----------------------------------------------------------------

bilstm_status logprob_sizes(const char *call, const bilstm_logprobs_args *args) {
    if (args == nullptr) return fail(BILSTM_INVALID_ARGUMENT, "%s: args is NULL", call);
    BL_CHECK(check_type(call, args->type));
    if (args->vocabulary == 0) return fail(BILSTM_INVALID_ARGUMENT, "%s: vocabulary is 0", call);
    if (args->rows > kMostRows || args->vocabulary > (1u << 20)) {
        return fail(BILSTM_DIMENSION_OVERFLOW, "%s: %llu rows of %u tokens exceed the kernel's indexing", call,
                    static_cast<unsigned long long>(args->rows), args->vocabulary);
    }
    if (args->top > static_cast<uint32_t>(kMostTop) || args->top > args->vocabulary) {
        return fail(BILSTM_INVALID_ARGUMENT, "%s: top is %u: at most %d and the vocabulary", call, args->top, kMostTop);
    }
    return BILSTM_OK;
}

bilstm_status logprobs(const char *call, const bilstm_logprobs_args *args, void *stream) {
    BL_CHECK(logprob_sizes(call, args));
    const bilstm_logprobs_args &a = *args;
    if (a.reserved != 0) return fail(BILSTM_INVALID_ARGUMENT, "%s: reserved must be 0", call);
    if (a.given > 1024) return fail(BILSTM_INVALID_ARGUMENT, "%s: %u given tokens a row: at most 1024", call, a.given);
    if (a.rows == 0) return BILSTM_OK;
    const uint64_t size = size_of(a.type);
    BL_CHECK(check_rows(call, "logits", a.logits, a.rows, a.vocabulary, size));
    if (a.given > 0) {
        BL_CHECK(check_buffer(call, "tokens", a.tokens, a.rows * a.given, 8, false));
        BL_CHECK(check_buffer(call, "logprobs", a.logprobs, a.rows * a.given, 4, false));
    }
    BL_CHECK(check_buffer(call, "entropy", a.entropy, a.rows, 4, false));
    if (a.top > 0) {
        BL_CHECK(check_buffer(call, "top_tokens", a.top_tokens, a.rows * a.top, 8, false));
        BL_CHECK(check_buffer(call, "top_logprobs", a.top_logprobs, a.rows * a.top, 4, false));
    }
    const uint64_t need = logprob_scratch_bytes(static_cast<int>(a.rows), static_cast<int>(a.vocabulary),
                                                static_cast<int>(a.top), elem_of(a.type));
    if (need > 0) {
        BL_CHECK(check_pointer(call, "scratch", a.scratch.data, 16));
        if (a.scratch.len < need) {
            return fail(BILSTM_BUFFER_LENGTH, "%s: scratch: expected at least %llu bytes, got %llu", call,
                        static_cast<unsigned long long>(need), static_cast<unsigned long long>(a.scratch.len));
        }
    }
    const bilstm_buffer none = {nullptr, 0};
    struct Region {
        const char *name;
        Bytes bytes;
    };
    const Region ins[] = {{"logits", bytes_of(a.logits, a.rows, a.vocabulary, size)},
                          {"tokens", bytes_of(a.given > 0 ? a.tokens : none, 8)}};
    const Region outs[] = {{"logprobs", bytes_of(a.given > 0 ? a.logprobs : none, 4)},
                           {"entropy", bytes_of(a.entropy, 4)},
                           {"top_tokens", bytes_of(a.top > 0 ? a.top_tokens : none, 8)},
                           {"top_logprobs", bytes_of(a.top > 0 ? a.top_logprobs : none, 4)},
                           {"scratch", bytes_of(need > 0 ? a.scratch : none, 1)}};
    for (const Region &o : outs) {
        for (const Region &in : ins) BL_CHECK(check_apart(call, o.name, o.bytes, in.name, in.bytes));
        for (const Region &other : outs) {
            if (&other != &o) BL_CHECK(check_apart(call, o.name, o.bytes, other.name, other.bytes));
        }
    }
    LogprobArgs k;
    k.logits = a.logits.data;
    k.stride = a.logits.stride;
    k.tokens = static_cast<const long long *>(a.tokens.data);
    k.logprobs = static_cast<float *>(const_cast<void *>(a.logprobs.data));
    k.entropy = static_cast<float *>(const_cast<void *>(a.entropy.data));
    k.top_tokens = static_cast<long long *>(const_cast<void *>(a.top_tokens.data));
    k.top_logprobs = static_cast<float *>(const_cast<void *>(a.top_logprobs.data));
    k.scratch = const_cast<void *>(a.scratch.data);
    k.rows = static_cast<int>(a.rows);
    k.vocabulary = static_cast<int>(a.vocabulary);
    k.given = static_cast<int>(a.given);
    k.top = static_cast<int>(a.top);
    DeviceScope scope(a.device);
    BL_CHECK(scope.enter(call));
    return launched(call, launch_token_logprobs(k, elem_of(a.type), static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

bilstm_status bilstm_causal_conv(const bilstm_conv_args *args, void *stream) {
    return conv("causal_conv", args, false, stream);
}

bilstm_status bilstm_causal_conv_step(const bilstm_conv_args *args, void *stream) {
    return conv("causal_conv_step", args, true, stream);
}

bilstm_status bilstm_scan_scratch(const bilstm_scan_args *args, uint64_t *bytes) {
    ScanArgs k;
    BL_CHECK(scan_sizes("scan_scratch", args, false, &k));
    if (bytes == nullptr) return fail(BILSTM_INVALID_ARGUMENT, "scan_scratch: bytes is NULL");
    *bytes = scan_scratch_bytes(k);
    return BILSTM_OK;
}

bilstm_status bilstm_scan(const bilstm_scan_args *args, void *stream) { return scan("scan", args, false, stream); }

bilstm_status bilstm_scan_step(const bilstm_scan_args *args, void *stream) { return scan("scan_step", args, true, stream); }

bilstm_status bilstm_add_rms_norm(const bilstm_norm_args *args, void *stream) {
    return norm("add_rms_norm", args, stream);
}

bilstm_status bilstm_token_logprobs_scratch(const bilstm_logprobs_args *args, uint64_t *bytes) {
    BL_CHECK(logprob_sizes("token_logprobs_scratch", args));
    if (bytes == nullptr) return fail(BILSTM_INVALID_ARGUMENT, "token_logprobs_scratch: bytes is NULL");
    *bytes = logprob_scratch_bytes(static_cast<int>(args->rows), static_cast<int>(args->vocabulary),
                                   static_cast<int>(args->top), elem_of(args->type));
    return BILSTM_OK;
}

bilstm_status bilstm_token_logprobs(const bilstm_logprobs_args *args, void *stream) {
    return logprobs("token_logprobs", args, stream);
}

}  // extern "C"
