// lm_norm.hip -- groups divided by the root of their mean square, weighted and
// gated.
//
//   y = x / sqrt(mean x^2 + eps) w silu(z),  or the same of x silu(z) without a gate
//
// Bound by HBM: x and z read once, y written once.  A group stays in registers
// between its sum and its outputs (8 KEEP elements a thread, x and z; what is
// longer is read again, from the L2).  8192 x 32 x 128 in bf16 40 us, 5.0 TB/s, where
// a copy reaches 5.15; 64 x 5001 in f16 4 us, a launch and three trips to memory.
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
    if (L > 4)
        with(std::integral_constant<int, 0x141>{});     // half mirror
    if (L > 8)
        with(std::integral_constant<int, 0x140>{});     // row mirror
    return v;
}

// Pack i of a group of `dim` elements: those from 8 i on.  Every load is unconditional:
// packs beyond the end are the last one again, and where dim is no multiple of 8 the last
// one is loaded from an earlier start.  The first `skip` elements are not its own.
// WHOLE: dim is a multiple of 8; SHORT: below 8, one pack with its elements at its end.
enum Shape { WHOLE, ODD, SHORT };
template <class T> struct Part8 {
    Pack<T, 8> v;
    int start, skip;
};
template <class T, Shape S> __device__ __forceinline__ Part8<T> part_of(const typename T::raw *p, int i, int dim)
{
    Part8<T> r;
    r.start = 8 * i < dim - 8 ? 8 * i : dim - 8;
    r.skip = 8 * i - r.start;
    if (S != SHORT) {
        r.v = load_pack<T, 8>(p + r.start);
    } else {
#pragma unroll
        for (int v = 0; v < 8; ++v)
            r.v.v[v] = p[r.start + v > 0 ? r.start + v : 0];
        r.skip = i == 0 ? -r.start : 8;
    }
    return r;
}

// THREADS share a group; a thread's k-th pack is pack threadIdx + THREADS k of 8
// elements.
template <class T, int THREADS, int KEEP, Shape S>
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
    const uint32_t *w = (const uint32_t *)a.weight + group * a.d.weight_group_stride;
    const int dim = (int)a.d.dim, packs = (dim + 7) / 8;
    const bool gated = a.z != nullptr, first = a.d.gate_first;

    using Part = Part8<T>;
    auto at = [&](const raw *p, int i) { return part_of<T, S>(p, i, dim); };
    // x, or x silu(z), of a pack
    auto values = [&](const Part &p, const Part &g, float (&f)[8]) {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            f[v] = T::load(p.v.v[v]);
            if (first)
                f[v] *= silu(T::load(g.v.v[v]));
        }
    };
    float sum = 0.0f;
    auto add = [&](const Part &p, const Part &g) {
        float f[8];
        values(p, g, f);
#pragma unroll
        for (int v = 0; v < 8; ++v)
            f[v] = S == WHOLE || v >= p.skip ? f[v] * f[v] : 0.0f;
        const float some = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        sum += S != WHOLE || p.skip == 0 ? some : 0.0f;
    };
    // A single pack's weights before the sum too: 262144 x 128 in bf16 38.3 us against
    // 40.2, 65536 x 512 39.1 and 41.0.  Of two packs, where lanes may have one, not:
    // 246723 x 136 62 us against 56.
    constexpr bool EARLY = KEEP == 1;
    float weights[8];
    auto weights_of = [&](const Part &p, float (&weight)[8]) {
        if (S != SHORT) {
            __builtin_memcpy(weight, w + p.start, sizeof(weight));
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                weight[v] = __uint_as_float(w[p.start + v > 0 ? p.start + v : 0]);
        }
    };
    Part keep[KEEP], gate[KEEP];
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        keep[k] = at(x, lane + THREADS * k);
        gate[k] = gated ? at(z, lane + THREADS * k) : keep[k];
        if (EARLY)
            weights_of(keep[k], weights);
    }
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        add(keep[k], gate[k]);
    for (int i = lane + THREADS * KEEP; i < packs; i += THREADS)
        add(at(x, i), at(z, i));
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
    auto put = [&](const Part &p, const Part &g, const float (&weight)[8]) {
        if (p.skip >= 8)
            return;
        float f[8];
        values(p, g, f);
        Pack<T, 8> out;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            float o = f[v] * r * weight[v];
            if (gated && !first)
                o *= silu(T::load(g.v.v[v]));
            out.v[v] = T::store(o);
        }
        if (S == WHOLE || p.skip == 0) {
            store_pack<T, 8>(y + p.start, out);
        } else {
#pragma unroll
            for (int v = 1; v < 8; ++v)
                if (v >= p.skip)
                    y[p.start + v] = out.v[v];
        }
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        if (!EARLY)
            weights_of(keep[k], weights);
        put(keep[k], gate[k], weights);
    }
    for (int i = lane + THREADS * KEEP; i < packs; i += THREADS) {
        const Part p = at(x, i), g = at(z, i);
        weights_of(p, weights);
        put(p, g, weights);
    }
}

template <class T, int THREADS, int KEEP> static int norm_groups_go(const NormArgs &a, hipStream_t s)
{
    constexpr int EACH = THREADS < 256 ? 256 / THREADS : 1;
    const uint64_t blocks = ((uint64_t)a.d.rows * a.d.groups + EACH - 1) / EACH;
    if ((__int128)a.d.rows * a.d.groups > 0xFFFFFFFFu || !launchable(blocks, THREADS * EACH))
        return (int)hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)blocks), block(THREADS * EACH);
    if (a.d.dim % 8 == 0)
        norm_kernel<T, THREADS, KEEP, WHOLE><<<grid, block, 0, s>>>(a);
    else if (THREADS > 4 || a.d.dim >= 8)
        norm_kernel<T, THREADS, KEEP, ODD><<<grid, block, 0, s>>>(a);
    else
        norm_kernel<T, 4, 1, SHORT><<<grid, block, 0, s>>>(a);
    return (int)hipGetLastError();
}

// The fewest threads that hold a group in one pack each, or in two.  bf16 (f32), 2^25
// elements, the time taken against the next best: 32 elements 4 threads 46 (79) us
// against 16's 128 (125); 64 elements 8 threads 38 (75); 128 elements 16 threads 40 (80)
// against 64's 49 (81); 256 elements two packs of 16 threads 40 (80) against 64's 69
// (78); 512 elements 64 threads 39 (75) against four packs of 16 48 (88); 1024 elements
// two packs of 64 threads 40 (79) against 256's 61 (74), and 520 elements 56 (81) against
// 111 (120); 2048 elements 256 threads 40 (72) against four packs of 64 47 (89); 4096
// elements two packs of 256 threads 40 (77) against 1024's 63 (84); 8192 elements 1024
// threads 39 (74) against four packs of 256 48 (87), and 16384 elements, half of them read
// twice, 44 (90) against 51 (106).  Few groups of 513 to 1024 elements take 256 threads,
// as the chip has compute units to spare: 64 x 1024 3.1 us against 4.2; 1000 x 1024 4.3
// and 4.4.
template <class T> static int norm_go(const NormArgs &a, hipStream_t s)
{
    if (a.d.dim <= 32)
        return norm_groups_go<T, 4, 1>(a, s);
    if (a.d.dim <= 64)
        return norm_groups_go<T, 8, 1>(a, s);
    if (a.d.dim <= 128)
        return norm_groups_go<T, 16, 1>(a, s);
    if (a.d.dim <= 256)
        return norm_groups_go<T, 16, 2>(a, s);
    if (a.d.dim <= 512)
        return norm_groups_go<T, 64, 1>(a, s);
    if (a.d.dim <= 1024 && a.d.rows * a.d.groups > 1024)
        return norm_groups_go<T, 64, 2>(a, s);
    if (a.d.dim <= 2048)
        return norm_groups_go<T, 256, 1>(a, s);
    return a.d.dim <= 4096 ? norm_groups_go<T, 256, 2>(a, s) : norm_groups_go<T, 1024, 1>(a, s);
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
