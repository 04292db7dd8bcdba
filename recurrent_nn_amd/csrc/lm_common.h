// lm_common.h -- shared by the language-model operators (convolution, scan,
// 8-bit projection, token scores): element types in memory, the arguments of
// each launch and the launch functions that lm_run.cpp calls.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/recurrent_nn_amd.h"

namespace rnnamd {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// Elements.  A stored value is raw bits (F32 uint32_t, BF16 and F16 uint16_t)
// widened to float32 on load; stores round to nearest even.
// ---------------------------------------------------------------------------

struct F32 {
    using raw = uint32_t;
    static __device__ __forceinline__ float load(raw r) { return __uint_as_float(r); }
    static __device__ __forceinline__ raw store(float v) { return __float_as_uint(v); }
};
struct BF16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(raw r) { return __uint_as_float((uint32_t)r << 16); }
    static __device__ __forceinline__ raw store(float v)
    {
        return __builtin_bit_cast(uint16_t, (__bf16)v);      // one conversion instruction
    }
};
struct F16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(raw r)
    {
        return (float)__builtin_bit_cast(_Float16, r);
    }
    static __device__ __forceinline__ raw store(float v)
    {
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
};

// N consecutive elements as one value for the widest loads and stores.
template <class T, int N> struct alignas((sizeof(typename T::raw) * N) < 16
                                             ? sizeof(typename T::raw) * N
                                             : 16) Pack {
    typename T::raw v[N];
};

// silu(v) = v / (1 + exp(-v)); the exponential in base 2, one reciprocal.
__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// ---------------------------------------------------------------------------
// Launch arguments
// ---------------------------------------------------------------------------

struct ConvArgs {
    rnn_conv_desc d;
    const void *x, *state_in;
    const float *weight, *bias;
    const int32_t *lens;
    void *y, *state_out;
};

struct ScanArgs {
    rnn_scan_desc d;
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias, *state_in;
    const int32_t *lens;
    void *y, *workspace;
    float *state_out;
};

struct QuantizeArgs {
    int64_t rows, cols, x_stride, q_stride;
    int32_t dtype;
    const void *x;
    int8_t *q;
    float *scale;
};

struct ProjectArgs {
    rnn_quant_desc d;
    const void *x;
    const float *x_scale, *w_scale, *bias;
    const int8_t *w;
    void *y, *workspace;
};

struct ScoresArgs {
    rnn_scores_desc d;
    const void *logits, *tokens;
    float *logprob, *entropy, *top_logprobs;
    int32_t *rank, *top_ids;
    void *workspace;
};

// Each returns a hipError_t as int; sizes have been checked and are not zero.
int launch_conv(const ConvArgs &a, hipStream_t s);
size_t scan_workspace(const rnn_scan_desc &d);
int launch_scan(const ScanArgs &a, hipStream_t s);
int launch_quantize(const QuantizeArgs &a, hipStream_t s);
size_t project_workspace(const rnn_quant_desc &d);
int launch_project(const ProjectArgs &a, hipStream_t s);
size_t scores_workspace(const rnn_scores_desc &d);
int launch_scores(const ScoresArgs &a, hipStream_t s);

}  // namespace rnnamd
