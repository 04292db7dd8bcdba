// lm_quant.hip -- rows to 8-bit integers with one scale each.
//
//   m = max|x|, r = 127 / m, q = rint(x r), scale = m / 127
//
// Bound by HBM: x read once, q written once.  A row stays in registers between
// its maximum and its rounding (up to 32 elements a thread; what is longer is
// read again, from the L2).  A wave takes a short row by itself, so that no
// barrier is needed; longer ones take a workgroup.  8192 x 4096 in bf16: 18.3 us,
// 5.5 TB/s.
#include "lm_common.h"

namespace rnnamd {

// THREADS (64 or 256) share a row; a thread's k-th pack is pack threadIdx +
// THREADS k of 8 elements.
template <class T, int THREADS>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs a)
{
    using raw = typename T::raw;
    constexpr int KEEP = 4;
    __shared__ uint32_t part[4];
    const int lane = threadIdx.x % THREADS;
    const int64_t row = THREADS == 64 ? (int64_t)blockIdx.x * 4 + threadIdx.x / 64 : blockIdx.x;
    if (THREADS == 64 && row >= a.rows)
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
    most = wave_max(most);
    if (THREADS > 64) {
        if (threadIdx.x % 64 == 0)
            part[threadIdx.x / 64] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
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

template <class T> static void quantize_go(const QuantizeArgs &a, hipStream_t s)
{
    // up to 2048 elements fit one wave's registers
    if (a.cols <= 2048)
        quantize_kernel<T, 64><<<dim3((uint32_t)((a.rows + 3) / 4)), dim3(256), 0, s>>>(a);
    else
        quantize_kernel<T, 256><<<dim3((uint32_t)a.rows), dim3(256), 0, s>>>(a);
}

int launch_quantize(const QuantizeArgs &a, hipStream_t s)
{
    switch (a.dtype) {
    case RNN_DTYPE_F32: quantize_go<F32>(a, s); break;
    case RNN_DTYPE_BF16: quantize_go<BF16>(a, s); break;
    default: quantize_go<F16>(a, s); break;
    }
    return (int)hipGetLastError();
}

}  // namespace rnnamd
