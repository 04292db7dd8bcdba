// lm_checks.h -- what the entry points of the language-model operators share:
// their errors and the checks made before anything is enqueued.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <new>
#include <string>

#include "common.h"

namespace rnnamd {

// What a check throws; nothing of it leaves the C entry points.
struct Fault {
    rnn_status status;
    std::string text;
};

[[noreturn]] inline void invalid(const std::string &text) { throw Fault{RNN_ERR_INVALID_INPUT, text}; }
[[noreturn]] inline void unsupported(const std::string &text) { throw Fault{RNN_ERR_UNSUPPORTED, text}; }

template <class F> rnn_status entry(const char *name, F &&body) noexcept
{
    try {
        set_error("");
        try {
            body();
            return RNN_OK;
        } catch (const Fault &f) {
            set_error(std::string(name) + ": " + f.text);
            return f.status;
        }
    } catch (...) {
        return RNN_ERR_OUT_OF_MEMORY;
    }
}

inline void launched(int rc)
{
    if (rc == (int)hipErrorInvalidConfiguration)
        unsupported("more work than one launch takes");
    if (rc)
        throw Fault{RNN_ERR_DEVICE, hipGetErrorString((hipError_t)rc)};
}

inline int64_t elem_size(int32_t dtype) { return dtype == RNN_DTYPE_F32 ? 4 : 2; }

inline void float_type(const char *name, int32_t dtype)
{
    if (dtype != RNN_DTYPE_F32 && dtype != RNN_DTYPE_BF16 && dtype != RNN_DTYPE_F16)
        invalid(std::string(name) + " must be RNN_DTYPE_F32, BF16 or F16");
}

inline void size_of(const char *name, int64_t v, int64_t lo = 0)
{
    if (v < lo || v > (int64_t)1 << 40)
        invalid(std::string(name) + " out of range: " + std::to_string(v));
}

inline void pointer(const char *name, const void *p, int64_t align, bool required = true)
{
    if (!p) {
        if (required)
            invalid(std::string(name) + " is required");
        return;
    }
    if ((uintptr_t)p % (uintptr_t)align)
        invalid(std::string(name) + " must be " + std::to_string(align) + "-byte aligned");
}

inline void workspace_of(const void *ws, size_t have, size_t need)
{
    if (need == 0)
        return;
    if (!ws || have < need)
        invalid("workspace missing or too small: " + std::to_string(need) + " bytes needed");
    if ((uintptr_t)ws % 256)
        invalid("workspace must be 256-byte aligned");
}

// Strides of a [n0, n1, inner] tensor: not negative, the extent countable; an
// output's elements must all be distinct.
inline void strides(const char *name, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner,
             bool output = false)
{
    if (n0 == 0 || n1 == 0 || inner == 0)
        return;
    const int64_t most = (int64_t)1 << 48;
    __int128 last = inner;
    if (n0 > 1)
        last += (__int128)(n0 - 1) * s0;
    if (n1 > 1)
        last += (__int128)(n1 - 1) * s1;
    if ((n0 > 1 && s0 < 0) || (n1 > 1 && s1 < 0) || last > most)
        invalid(std::string(name) + ": stride out of range");
    if (!output)
        return;
    const bool swap = n0 > 1 && n1 > 1 && s0 < s1;
    const int64_t in_n = swap ? n0 : n1, in_s = swap ? s0 : s1;
    const int64_t out_n = swap ? n1 : n0, out_s = swap ? s1 : s0;
    const int64_t span = in_n > 1 ? (in_n - 1) * in_s + inner : inner;
    if ((in_n > 1 && in_s < inner) || (out_n > 1 && out_s < span))
        invalid(std::string(name) + ": strides make its elements overlap");
}

inline void not_on(const char *out, const void *p, const char *in, const void *q)
{
    if (p && p == q)
        invalid(std::string(out) + " must not be " + in);
}

}  // namespace rnnamd
