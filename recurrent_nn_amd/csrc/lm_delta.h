// lm_delta.h -- shared by the two forms of the gated delta rule (single steps,
// chunks): gates, lengths and the choice between the forms.
#pragma once

#include "lm_common.h"

namespace rnnamd {

// log of the decay from what g holds, within [-104, 0] (e^-104 is 0 in float32).
// A sum of them over a chunk stays finite, and NaN stays NaN.
__device__ __forceinline__ float log_decay(float g, bool through_A, float A, float bias)
{
    float a = g;
    if (through_A) {
        const float x = g + bias;
        a = A * (__builtin_fmaxf(x, 0.0f) + log1pf(expf(-__builtin_fabsf(x))));
    }
    a = a > 0.0f ? 0.0f : a;
    return a < -104.0f ? -104.0f : a;
}
__device__ __forceinline__ float rate_of(float beta, bool sigmoid)
{
    return sigmoid ? 1.0f / (1.0f + expf(-beta)) : beta;
}
template <class T> __device__ __forceinline__ float gate_at(const void *p, int32_t dtype, int64_t i)
{
    return dtype == RNN_DTYPE_F32 ? ((const float *)p)[i] : T::load(((const typename T::raw *)p)[i]);
}
__device__ __forceinline__ int delta_steps(const DeltaArgs &a, int64_t b)
{
    int n = (int)a.d.steps;
    if (a.lens) {
        const int l = a.lens[b];
        n = l < 0 ? 0 : l < n ? l : n;
    }
    return n;
}
__device__ __forceinline__ float key_scale(float squares, int32_t normalize)
{
    return normalize ? 1.0f / sqrtf(squares + RNN_DELTA_KEY_EPS) : 1.0f;
}

// Chunks of 64 steps (lm_delta_chunk.hip); sizes are not zero.
size_t delta_chunks_workspace(const rnn_delta_desc &d);
int launch_delta_chunks(const DeltaArgs &a, hipStream_t s);

}  // namespace rnnamd
