// lm_norm.hip -- groups divided by the root of their mean square, weighted and
// gated.
//
//   y = x / sqrt(mean x^2 + eps) w silu(z),  or the same of x silu(z) without a gate
//
// Bound by HBM: x and z read once, y written once.  A group stays in registers
// between its sum and its outputs (8 KEEP elements a thread, x and z; what is
// longer is read again, from the L2).
#include <type_traits>

#include "lm_common.h"

namespace rnnamd {

// The sum over L adjacent lanes, in all of them.
template <int L> __device__ __forceinline__ float lanes_sum(float v)
{
    if (L >= 64)
        return wave_sum(v);
    auto with = [&](auto ctrl) {
        v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
            0, (int)__float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    with(std::integral_constant<int, 0xB1>{});          // lane xor 1
    with(std::integral_constant<int, 0x4E>{});          // lane xor 2
    if (L > 4) {
        with(std::integral_constant<int, 0x141>{});     // half mirror
        with(std::integral_constant<int, 0x140>{});     // row mirror
    }
    return v;
}

// THREADS share a group; a thread's k-th pack is pack threadIdx + THREADS k of 8
// elements.
template <class T, int THREADS, int KEEP>
__global__ __launch_bounds__(THREADS > 256 ? THREADS : 256) void norm_kernel(NormArgs a)
{
    using raw = typename T::raw;
    constexpr int EACH = THREADS < 256 ? 256 / THREADS : 1, WAVES = THREADS / 64;
    __shared__ float part[WAVES > 1 ? WAVES : 1];
    const int lane = threadIdx.x % THREADS;
    const uint32_t id = blockIdx.x * EACH + threadIdx.x / THREADS;
    const uint32_t row = id / (uint32_t)a.d.groups, group = id % (uint32_t)a.d.groups;
    if (row >= a.d.rows)
        return;
    const raw *x = (const raw *)a.x + row * a.d.x_row_stride + group * a.d.x_group_stride;
    const raw *z = a.z ? (const raw *)a.z + row * a.d.z_row_stride + group * a.d.z_group_stride : x;
    raw *y = (raw *)a.y + row * a.d.y_row_stride + group * a.d.y_group_stride;
    const float *w = a.weight + group * a.d.weight_group_stride;
    const int dim = (int)a.d.dim, packs = (dim + 7) / 8;
    const bool gated = a.z != nullptr, first = a.d.gate_first;

    auto pack = [&](const raw *p, int i) {
        Pack<T, 8> r{};
        if (8 * i + 8 <= dim) {
            r = load_pack<T, 8>(p + 8 * i);
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                if (8 * i + v < dim)
                    r.v[v] = p[8 * i + v];
        }
        return r;
    };
    auto value = [&](const Pack<T, 8> &p, const Pack<T, 8> &g, int v) {
        const float f = T::load(p.v[v]);
        return first ? f * silu(T::load(g.v[v])) : f;
    };
    float sum = 0.0f;
    auto add = [&](const Pack<T, 8> &p, const Pack<T, 8> &g) {
        float f[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            f[v] = value(p, g, v);
            f[v] *= f[v];
        }
        sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    };
    Pack<T, 8> keep[KEEP], gate[KEEP];
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        keep[k] = pack(x, lane + THREADS * k);
        gate[k] = keep[k];
        if (gated)
            gate[k] = pack(z, lane + THREADS * k);
    }
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        add(keep[k], gate[k]);
    for (int i = lane + THREADS * KEEP; i < packs; i += THREADS)
        add(pack(x, i), pack(z, i));
    sum = lanes_sum<THREADS < 64 ? THREADS : 64>(sum);
    if (THREADS > 64) {
        if (threadIdx.x % 64 == 0)
            part[threadIdx.x / 64] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i)
            sum += part[i];
    }
    const float r = 1.0f / sqrtf(sum / (float)dim + a.d.eps);
    auto put = [&](int i, const Pack<T, 8> &p, const Pack<T, 8> &g) {
        auto one = [&](int v, float weight) {
            const float f = value(p, g, v) * r * weight;
            return T::store(gated && !first ? f * silu(T::load(g.v[v])) : f);
        };
        if (8 * i + 8 <= dim) {
            const Pack<F32, 8> weight = load_pack<F32, 8>((const uint32_t *)w + 8 * i);
            Pack<T, 8> out;
#pragma unroll
            for (int v = 0; v < 8; ++v)
                out.v[v] = one(v, F32::load(weight.v[v]));
            store_pack<T, 8>(y + 8 * i, out);
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                if (8 * i + v < dim)
                    y[8 * i + v] = one(v, w[8 * i + v]);
        }
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        put(lane + THREADS * k, keep[k], gate[k]);
    for (int i = lane + THREADS * KEEP; i < packs; i += THREADS)
        put(i, pack(x, i), pack(z, i));
}

template <class T, int THREADS, int KEEP> static int norm_groups_go(const NormArgs &a, hipStream_t s)
{
    constexpr int EACH = THREADS < 256 ? 256 / THREADS : 1;
    const uint64_t blocks = ((uint64_t)a.d.rows * a.d.groups + EACH - 1) / EACH;
    if ((__int128)a.d.rows * a.d.groups > 0xFFFFFFFFu || !launchable(blocks, THREADS * EACH))
        return (int)hipErrorInvalidConfiguration;
    norm_kernel<T, THREADS, KEEP><<<dim3((uint32_t)blocks), dim3(THREADS * EACH), 0, s>>>(a);
    return (int)hipGetLastError();
}

template <class T> static int norm_go(const NormArgs &a, hipStream_t s)
{
    if (a.d.dim <= 32)
        return norm_groups_go<T, 4, 1>(a, s);
    if (a.d.dim <= 256)
        return norm_groups_go<T, 16, 2>(a, s);
    if (a.d.dim <= 2048)
        return norm_groups_go<T, 64, 4>(a, s);
    return a.d.dim <= 8192 ? norm_groups_go<T, 256, 4>(a, s) : norm_groups_go<T, 1024, 4>(a, s);
}

int launch_norm(const NormArgs &a, hipStream_t s)
{
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: return norm_go<F32>(a, s);
    case RNN_DTYPE_BF16: return norm_go<BF16>(a, s);
    default: return norm_go<F16>(a, s);
    }
}

}  // namespace rnnamd
