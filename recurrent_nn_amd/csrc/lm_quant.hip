// lm_quant.hip -- rows to 8-bit integers with one scale each.
//
//   m = max|x|, r = 127 / m, q = rint(x r), scale = m / 127
//
// Bound by HBM: x read once, q written once.  A row stays in registers between
// its maximum and its rounding (up to 32 elements a thread; what is longer is
// read again, from the L2).  4, 16 or 64 lanes take a short row, so that no
// barrier is needed and lanes without elements are few; longer ones take a
// workgroup.  8192 x 4096 in bf16: 17.7 us, 5.7 TB/s.
#include <type_traits>

#include "lm_common.h"

namespace rnnamd {

// The maximum over L adjacent lanes, in all of them.
template <int L> __device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    if (L >= 64)
        return wave_max(v);
    auto with = [&](auto ctrl) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF,
                                                                 0xF, true);
        v = o > v ? o : v;
    };
    with(std::integral_constant<int, 0xB1>{});          // lane xor 1
    with(std::integral_constant<int, 0x4E>{});          // lane xor 2
    if (L > 4) {
        with(std::integral_constant<int, 0x141>{});     // half mirror
        with(std::integral_constant<int, 0x140>{});     // row mirror
    }
    return v;
}

// THREADS share a row; a thread's k-th pack is pack threadIdx + THREADS k of 8
// elements.
template <class T, int THREADS>
__global__ __launch_bounds__(THREADS > 256 ? THREADS : 256) void quantize_kernel(QuantizeArgs a)
{
    using raw = typename T::raw;
    constexpr int KEEP = 4;
    constexpr int ROWS = THREADS < 256 ? 256 / THREADS : 1, WAVES = THREADS / 64;
    __shared__ uint32_t part[WAVES > 1 ? WAVES : 1];
    const int lane = threadIdx.x % THREADS;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS;
    if (row >= a.rows)
        return;
    const raw *x = (const raw *)a.x + row * a.x_stride;
    const int cols = (int)a.cols;

    auto pack = [&](int i) {
        Pack<T, 8> p{};
        if (8 * i + 8 <= cols) {
            p = load_pack<T, 8>(x + 8 * i);
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                if (8 * i + v < cols)
                    p.v[v] = x[8 * i + v];
        }
        return p;
    };
    const int packs = (cols + 7) / 8, out_packs = (int)(a.q_stride / 8);
    Pack<T, 8> keep[KEEP];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        keep[k] = pack(lane + THREADS * k);
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        most = pack_max<T, 8>(keep[k], most);
    for (int i = lane + THREADS * KEEP; i < packs; i += THREADS)
        most = pack_max<T, 8>(pack(i), most);
    most = lanes_max<THREADS>(most);
    if (THREADS > 64) {
        if (threadIdx.x % 64 == 0)
            part[threadIdx.x / 64] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i)
            most = part[i] > most ? part[i] : most;
    }
    const RowScale rs = row_scale(__uint_as_float(most), most < kInfBits);
    int8_t *q = a.q + row * a.q_stride;
    auto put = [&](int i, const Pack<T, 8> &p) {
        if (i < out_packs)
            *(uint2 *)(q + 8 * i) = pack_8bit<T>(p, rs.factor);
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        put(lane + THREADS * k, keep[k]);
    for (int i = lane + THREADS * KEEP; i < out_packs; i += THREADS)
        put(i, pack(i));
    if (lane == 0)
        a.scale[row] = rs.scale;
}

template <class T, int THREADS> static int quantize_rows_go(const QuantizeArgs &a, hipStream_t s)
{
    constexpr int ROWS = THREADS < 256 ? 256 / THREADS : 1;
    const int64_t blocks = (a.rows + ROWS - 1) / ROWS;
    if (!launchable(blocks, THREADS * ROWS))
        return (int)hipErrorInvalidConfiguration;
    quantize_kernel<T, THREADS><<<dim3((uint32_t)blocks), dim3(THREADS * ROWS), 0, s>>>(a);
    return (int)hipGetLastError();
}

// The fewest threads whose registers (32 elements each) hold a row: 100000 x 100
// in bf16 takes 4 lanes a row 10.5 us, a wave 44 us; 16384 x 512 by 16 lanes 6.3 us,
// a wave 10.2 us.  1024 threads only where they read ahead of the row's second
// reading (300 x 100000: 23.5 us, 256 threads 45.5 us); 2000 x 9000 fits them and
// takes 18.4 us, 256 threads 12.6 us.
template <class T> static int quantize_go(const QuantizeArgs &a, hipStream_t s)
{
    if (a.cols <= 128)
        return quantize_rows_go<T, 4>(a, s);
    if (a.cols <= 512)
        return quantize_rows_go<T, 16>(a, s);
    if (a.cols <= 2048)
        return quantize_rows_go<T, 64>(a, s);
    return a.cols <= 32768 ? quantize_rows_go<T, 256>(a, s) : quantize_rows_go<T, 1024>(a, s);
}

int launch_quantize(const QuantizeArgs &a, hipStream_t s)
{
    switch (a.dtype) {
    case RNN_DTYPE_F32: return quantize_go<F32>(a, s);
    case RNN_DTYPE_BF16: return quantize_go<BF16>(a, s);
    default: return quantize_go<F16>(a, s);
    }
}

}  // namespace rnnamd
