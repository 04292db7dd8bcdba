// lm_scan.hip -- selective state space scan.
//
//   s = softplus(dt + dt_bias);  h[n] = exp(s A[n]) h[n] + s x B[n]
//   y = (sum_n C[n] h[n] + D x) silu(z)
//
// First form: a group of lanes as wide as the states (rounded up to a power
// of two) holds one channel's state, one value a lane, and walks the steps.
#include "lm_common.h"

namespace rnnamd {

// log(1 + exp(v)) = max(v, 0) + log1p(w), w = exp(-|v|) in (0, 1].  With
// q = w / (2 + w), log1p(w) = 2 atanh(q) = 2 q (1 + q^2/3 + q^4/5 + ...): no
// cancellation for small w; q <= 1/3, so nine terms reach 2^-29.
__device__ __forceinline__ float softplus(float v)
{
    const float w = __builtin_amdgcn_exp2f(-__builtin_fabsf(v) * kLog2e);
    const float q = w * __builtin_amdgcn_rcpf(2.0f + w);
    const float r = q * q;
    float p = 1.0f / 17.0f;
    p = __builtin_fmaf(p, r, 1.0f / 15.0f);
    p = __builtin_fmaf(p, r, 1.0f / 13.0f);
    p = __builtin_fmaf(p, r, 1.0f / 11.0f);
    p = __builtin_fmaf(p, r, 1.0f / 9.0f);
    p = __builtin_fmaf(p, r, 1.0f / 7.0f);
    p = __builtin_fmaf(p, r, 1.0f / 5.0f);
    p = __builtin_fmaf(p, r, 1.0f / 3.0f);
    p = __builtin_fmaf(p, r, 1.0f);
    const float l = __builtin_fmaf(q + q, p, v > 0.0f ? v : 0.0f);
    return v != v ? v : l;
}

template <class T> __global__ __launch_bounds__(256) void scan_kernel(ScanArgs a, int32_t width)
{
    using raw = typename T::raw;
    const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / width;
    const int32_t n = threadIdx.x % width;
    const int64_t b = id / a.d.dim, c = id % a.d.dim;
    if (b >= a.d.batch)
        return;
    const int64_t steps = a.d.steps, N = a.d.states;
    int64_t len = steps;
    if (a.lens) {
        const int64_t l = a.lens[b];
        len = l < 0 ? 0 : (l < steps ? l : steps);
    }
    const bool on = n < N;
    const int64_t g = c / (a.d.dim / a.d.groups);
    const float A = on && len > 0 ? a.A[c * N + n] * kLog2e : 0.0f;
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f;
    const float D = a.D ? a.D[c] : 0.0f;
    float h = on && a.state_in ? a.state_in[(b * a.d.dim + c) * N + n] : 0.0f;
    const raw *x = (const raw *)a.x + b * a.d.x_batch_stride + c;
    const raw *dt = (const raw *)a.dt + b * a.d.dt_batch_stride + c;
    const raw *z = a.z ? (const raw *)a.z + b * a.d.z_batch_stride + c : nullptr;
    const raw *B = (const raw *)a.B + b * a.d.B_batch_stride + g * a.d.B_group_stride + n;
    const raw *C = (const raw *)a.C + b * a.d.C_batch_stride + g * a.d.C_group_stride + n;
    raw *y = (raw *)a.y + b * a.d.y_batch_stride + c;
    for (int64_t t = 0; t < len; ++t) {
        const float xv = T::load(x[t * a.d.x_step_stride]);
        float s = T::load(dt[t * a.d.dt_step_stride]) + bias;
        if (a.d.dt_softplus)
            s = softplus(s);
        float p = 0.0f;
        if (on) {
            h = __builtin_fmaf(__builtin_amdgcn_exp2f(s * A), h,
                               (s * xv) * T::load(B[t * a.d.B_step_stride]));
            p = T::load(C[t * a.d.C_step_stride]) * h;
        }
        for (int m = width / 2; m > 0; m /= 2)
            p += __shfl_xor(p, m, 64);
        if (n == 0) {
            if (a.D)
                p = __builtin_fmaf(D, xv, p);
            if (z)
                p *= silu(T::load(z[t * a.d.z_step_stride]));
            y[t * a.d.y_step_stride] = T::store(p);
        }
    }
    if (n == 0)
        for (int64_t t = len; t < steps; ++t)
            y[t * a.d.y_step_stride] = T::store(0.0f);
    if (on && a.state_out)
        a.state_out[(b * a.d.dim + c) * N + n] = h;
}

size_t scan_workspace(const rnn_scan_desc &) { return 0; }

int launch_scan(const ScanArgs &a, hipStream_t s)
{
    int32_t width = 1;
    while (width < a.d.states)
        width *= 2;
    const int64_t blocks = (a.d.batch * a.d.dim * width + 255) / 256;
    if (blocks > 0x7fffffff)
        return (int)hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)blocks), block(256);
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: scan_kernel<F32><<<grid, block, 0, s>>>(a, width); break;
    case RNN_DTYPE_BF16: scan_kernel<BF16><<<grid, block, 0, s>>>(a, width); break;
    default: scan_kernel<F16><<<grid, block, 0, s>>>(a, width); break;
    }
    return (int)hipGetLastError();
}

}  // namespace rnnamd
