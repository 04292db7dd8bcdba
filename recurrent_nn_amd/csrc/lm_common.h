// lm_common.h -- shared by the language-model operators (convolution, scan,
// 8-bit projection, token scores): element types in memory, the arguments of
// each launch and the launch functions that lm_run.cpp calls.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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

// N consecutive elements at an address aligned to one of them (global memory
// takes wide accesses at any such address).
template <class T, int N> __device__ __forceinline__ Pack<T, N> load_pack(const typename T::raw *p)
{
    Pack<T, N> v;
    __builtin_memcpy(v.v, p, sizeof(v.v));
    return v;
}
template <class T, int N>
__device__ __forceinline__ void store_pack(typename T::raw *p, const Pack<T, N> &v)
{
    __builtin_memcpy(p, v.v, sizeof(v.v));
}

// Four elements as loaded, in whole words: taken apart where they are used, so
// that a loop can carry them while the load is in flight.
template <class T> struct Words4 {
    static constexpr int kWords = sizeof(typename T::raw);      // 4 elements: 2 or 4 words
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int v) const
    {
        if constexpr (kWords == 4)
            return T::load(w[v]);
        else
            return T::load((typename T::raw)(v % 2 ? w[v / 2] >> 16 : w[v / 2] & 0xFFFFu));
    }
    __device__ __forceinline__ void load(const typename T::raw *p) { __builtin_memcpy(w, p, sizeof(w)); }
    // Without the first `n` (0 to 3; else as it is, or of no meaning).
    __device__ __forceinline__ void drop(int n)
    {
        if constexpr (kWords == 4) {
            const uint32_t a = w[1], b = w[2], c = w[3];
            if (n > 0) {
                w[0] = n == 1 ? a : n == 2 ? b : c;
                w[1] = n == 1 ? b : c;
                w[2] = c;
            }
        } else {
            const uint64_t all = ((uint64_t)w[1] << 32 | w[0]) >> (n > 0 ? 16 * (n & 3) : 0);
            w[0] = (uint32_t)all;
            w[1] = (uint32_t)(all >> 32);
        }
    }
    __device__ __forceinline__ void set(int v, typename T::raw r)
    {
        if constexpr (kWords == 4)
            w[v] = r;
        else
            w[v / 2] = v % 2 ? w[v / 2] | (uint32_t)r << 16 : (uint32_t)r;
    }
};

// A row's factor to 8 bits and its scale.  max|x| below 2^-100 would bring
// factors near overflow: such a row counts as zero.
struct RowScale {
    float factor, scale;
};
__device__ __forceinline__ RowScale row_scale(float most, bool finite)
{
    if (!finite)
        return {0.0f, __uint_as_float(0x7FC00000u)};
    if (!(most >= 0x1p-100f))
        return {0.0f, 0.0f};
    return {127.0f / most, most / 127.0f};
}

// A value of the wave's 64 lanes together, in all of them: op(own, other) with
// other = `none` (which changes nothing) where a lane has no partner.
template <class F> __device__ __forceinline__ uint32_t over_wave(uint32_t v, uint32_t none, F op)
{
    auto with = [&](auto ctrl, auto rows) {
        v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, decltype(ctrl)::value,
                                                        decltype(rows)::value, 0xF, false));
    };
    with(std::integral_constant<int, 0xB1>{}, std::integral_constant<int, 0xF>{});    // lane xor 1
    with(std::integral_constant<int, 0x4E>{}, std::integral_constant<int, 0xF>{});    // lane xor 2
    with(std::integral_constant<int, 0x141>{}, std::integral_constant<int, 0xF>{});   // half mirror
    with(std::integral_constant<int, 0x140>{}, std::integral_constant<int, 0xF>{});   // row mirror
    with(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});   // row 0 to 1, 2 to 3
    with(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});   // rows 0, 1 to 2, 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// (Magnitudes order as their bits do, infinities and NaN above all finite ones.)
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    return over_wave(v, 0u, [](uint32_t a, uint32_t b) { return b > a ? b : a; });
}
__device__ __forceinline__ uint32_t wave_sum(uint32_t v)
{
    return over_wave(v, 0u, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ __forceinline__ float wave_sum(float v)
{
    return __uint_as_float(over_wave(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
constexpr uint32_t kInfBits = 0x7F800000u;

// Four values to four 8-bit integers in a word; a row without a factor (zero,
// or not finite) is 0.  |x factor| <= 127 (1 + 2^-23): rounds to 127 at most.  Added
// to 1.5 2^23, whose last place is 1, the product is rounded to an integer (half
// to even), and its two's complement is the sum's last bits.
__device__ __forceinline__ uint32_t to_8bit(float a, float b, float c, float d, float factor)
{
    auto one = [&](float v) { return __float_as_uint(v * factor + 0x1.8p23f); };
    const uint32_t low = __builtin_amdgcn_perm(one(b), one(a), 0x0C0C0400u);
    const uint32_t high = __builtin_amdgcn_perm(one(d), one(c), 0x04000C0Cu);
    return factor == 0.0f ? 0u : low | high;
}
template <class T> __device__ __forceinline__ uint2 pack_8bit(const Pack<T, 8> &p, float factor)
{
    return {to_8bit(T::load(p.v[0]), T::load(p.v[1]), T::load(p.v[2]), T::load(p.v[3]), factor),
            to_8bit(T::load(p.v[4]), T::load(p.v[5]), T::load(p.v[6]), T::load(p.v[7]), factor)};
}
template <class T, int N>
__device__ __forceinline__ uint32_t pack_max(const Pack<T, N> &p, uint32_t m)
{
#pragma unroll
    for (int v = 0; v < N; ++v) {
        const uint32_t u = __float_as_uint(T::load(p.v[v])) & 0x7FFFFFFFu;
        m = u > m ? u : m;
    }
    return m;
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

// Whether a launch can have so many workgroups: a grid's threads are counted in 32 bits.
inline bool launchable(uint64_t workgroups, uint32_t threads) { return workgroups <= 0xFFFFFFFFu / threads; }

// Each returns a hipError_t as int (hipErrorInvalidConfiguration, with nothing
// enqueued, for more than a launch takes); sizes have been checked and are not zero.
int launch_conv(const ConvArgs &a, hipStream_t s);
size_t scan_workspace(const rnn_scan_desc &d);
int launch_scan(const ScanArgs &a, hipStream_t s);
int launch_quantize(const QuantizeArgs &a, hipStream_t s);
size_t project_workspace(const rnn_quant_desc &d);
int launch_project(const ProjectArgs &a, hipStream_t s);
size_t scores_workspace(const rnn_scores_desc &d);
int launch_scores(const ScoresArgs &a, hipStream_t s);

}  // namespace rnnamd
