// lm_conv.hip -- causal convolution of each channel over its last `taps`
// inputs, with the window of earlier inputs carried as a state.
//
//   v[t] = bias + sum_{j < K} weight[j] xx[t + j],   xx = window, x
//
// Bound by HBM: x read once, y written once.  A thread owns VEC adjacent
// channels (8 bytes) and a run of steps: the last K - 1 inputs and the weights
// stay in registers, so an input is loaded once by the run that owns it and
// K - 1 times less by the next run (from the L2).  Eight bytes and not sixteen:
// half the registers, twice the waves, and the loads of eight steps of each in
// flight (8192 x 4096 in bf16: 28.2 us, 4.8 TB/s; with 16 bytes 37.4).
#include "lm_common.h"

namespace rnnamd {

// The first run of a batch row also writes the new window, after it has read
// the old one: the two may be the same memory.
template <class T, int K, int VEC>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs a, uint32_t slots, uint32_t runs,
                                                   uint32_t run_steps)
{
    using P = Pack<T, VEC>;
    using raw = typename T::raw;
    const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const uint32_t slot = (uint32_t)(id % slots);
    const uint64_t rest = id / slots;
    const uint32_t run = (uint32_t)(rest % runs);
    const int64_t b = (int64_t)(rest / runs);
    if (b >= a.d.batch)
        return;
    // the last slot of channels that VEC does not divide begins earlier
    const int64_t c = (int64_t)slot * VEC + VEC <= a.d.dim ? (int64_t)slot * VEC : a.d.dim - VEC;
    const int64_t steps = a.d.steps, dim = a.d.dim;
    const int64_t t0 = (int64_t)run * run_steps;
    const int64_t t1 = t0 + run_steps < steps ? t0 + run_steps : steps;
    int64_t len = steps;
    if (a.lens) {
        const int64_t l = a.lens[b];
        len = l < 0 ? 0 : (l < steps ? l : steps);
    }
    const raw *x = (const raw *)a.x + b * a.d.x_batch_stride + c;
    raw *y = (raw *)a.y + b * a.d.y_batch_stride + c;
    const raw *in = a.state_in ? (const raw *)a.state_in + b * (K - 1) * dim + c : nullptr;

    // input i of xx: the window first, then x
    auto input = [&](int64_t i) {
        P p{};
        if (i >= K - 1)
            p = load_pack<T, VEC>(x + (i - (K - 1)) * a.d.x_step_stride);
        else if (in)
            p = load_pack<T, VEC>(in + i * dim);
        return p;
    };

    const int64_t end = t1 < len ? t1 : len;
    if (t0 < end) {
        float w[K][VEC], bias[VEC], win[K][VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            bias[v] = a.bias ? a.bias[c + v] : 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j)
                w[j][v] = a.weight[(c + v) * K + j];
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const P p = input(t0 + j);
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                win[j][v] = T::load(p.v[v]);
        }
        // AHEAD inputs at a time, the next ones on their way meanwhile
        auto step = [&](const P &p, int64_t t) {
            P out;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                win[K - 1][v] = T::load(p.v[v]);
                float s = bias[v];
#pragma unroll
                for (int j = 0; j < K; ++j)
                    s = __builtin_fmaf(w[j][v], win[j][v], s);
                out.v[v] = T::store(a.d.silu ? silu(s) : s);
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    win[j][v] = win[j + 1][v];
            }
            store_pack<T, VEC>(y + t * a.d.y_step_stride, out);
        };
        constexpr int AHEAD = 8;
        int64_t t = t0;
        for (; t + AHEAD <= end; t += AHEAD) {
            P p[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                p[i] = load_pack<T, VEC>(x + (t + i) * a.d.x_step_stride);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                step(p[i], t + i);
        }
        for (; t < end; ++t)
            step(load_pack<T, VEC>(x + t * a.d.x_step_stride), t);
    }
    for (int64_t t = t0 > end ? t0 : end; t < t1; ++t)
        store_pack<T, VEC>(y + t * a.d.y_step_stride, P{});

    if (K > 1 && run == 0 && a.state_out) {
        P next[K - 1 > 0 ? K - 1 : 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            next[j] = input(len + j);
        raw *out = (raw *)a.state_out + b * (K - 1) * dim + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            store_pack<T, VEC>(out + j * dim, next[j]);
    }
}

template <class T, int K, int VEC> static int conv_go(const ConvArgs &a, hipStream_t s)
{
    const uint64_t slots = (uint64_t)((a.d.dim + VEC - 1) / VEC);
    // runs of up to 32 steps (the K - 1 inputs before a run are read twice),
    // shorter ones while the chip is not full; never less than K - 1, so that only
    // the first run, which may replace the window in place, reads it
    static_assert(K - 1 <= 8, "a run is as long as the window");
    uint64_t run_steps = 32;
    while (run_steps > 8 && slots * (uint64_t)a.d.batch *
                                (((uint64_t)a.d.steps + run_steps - 1) / run_steps) < 262144)
        run_steps /= 2;
    uint64_t runs = ((uint64_t)a.d.steps + run_steps - 1) / run_steps;
    if (runs == 0)
        runs = 1;
    const uint64_t blocks = (slots * runs * (uint64_t)a.d.batch + 255) / 256;
    if (!launchable(blocks, 256) || runs > 0xffffffffull || slots > 0xffffffffull)
        return (int)hipErrorInvalidConfiguration;
    conv_kernel<T, K, VEC><<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(
        a, (uint32_t)slots, (uint32_t)runs, (uint32_t)run_steps);
    return (int)hipGetLastError();
}

template <class T, int K> static int conv_vec(const ConvArgs &a, hipStream_t s)
{
    // Channels that two threads would share are none where the state is replaced
    // in place: one thread could read what the other has written.
    constexpr int V = 8 / sizeof(typename T::raw);
    const bool apart = !a.state_out || a.state_in != a.state_out;
    return a.d.dim % V == 0 || (a.d.dim > V && apart) ? conv_go<T, K, V>(a, s)
                                                      : conv_go<T, K, 1>(a, s);
}

template <class T> static int conv_taps(const ConvArgs &a, hipStream_t s)
{
    switch (a.d.taps) {
    case 1: return conv_vec<T, 1>(a, s);
    case 2: return conv_vec<T, 2>(a, s);
    case 3: return conv_vec<T, 3>(a, s);
    case 4: return conv_vec<T, 4>(a, s);
    case 5: return conv_vec<T, 5>(a, s);
    case 6: return conv_vec<T, 6>(a, s);
    case 7: return conv_vec<T, 7>(a, s);
    default: return conv_vec<T, 8>(a, s);
    }
}

int launch_conv(const ConvArgs &a, hipStream_t s)
{
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: return conv_taps<F32>(a, s);
    case RNN_DTYPE_BF16: return conv_taps<BF16>(a, s);
    default: return conv_taps<F16>(a, s);
    }
}

}  // namespace rnnamd
