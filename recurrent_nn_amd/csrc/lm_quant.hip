// lm_quant.hip -- rows to 8-bit integers with one scale each, and the matrix
// product of such rows.
//
//   m = max|x|, r = 127 / m, q = rint(x r), scale = m / 127
//   y[i,o] = (sum_k qx[i,k] w[o,k]) (x_scale[i] w_scale[o]) + bias[o]
#include "lm_common.h"

namespace rnnamd {

// A row's factor to 8 bits and its scale.  max|x| below 2^-100 would bring
// factors near overflow: such a row counts as zero.  (The comparison also
// sends NaN there; the caller has marked it.)
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

template <class T> __global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs a)
{
    using raw = typename T::raw;
    __shared__ float part[4];
    __shared__ int bad[4];
    const int64_t row = blockIdx.x;
    const raw *x = (const raw *)a.x + row * a.x_stride;
    float most = 0.0f;
    int nonfinite = 0;
    for (int64_t k = threadIdx.x; k < a.cols; k += 256) {
        const float v = __builtin_fabsf(T::load(x[k]));
        nonfinite |= !(v < __builtin_inff());
        most = v > most ? v : most;
    }
    for (int m = 32; m > 0; m /= 2) {
        const float o = __shfl_xor(most, m, 64);
        most = o > most ? o : most;
        nonfinite |= __shfl_xor(nonfinite, m, 64);
    }
    if (threadIdx.x % 64 == 0) {
        part[threadIdx.x / 64] = most;
        bad[threadIdx.x / 64] = nonfinite;
    }
    __syncthreads();
    for (int i = 0; i < 4; ++i) {
        most = part[i] > most ? part[i] : most;
        nonfinite |= bad[i];
    }
    const RowScale rs = row_scale(most, !nonfinite);
    int8_t *q = a.q + row * a.q_stride;
    for (int64_t k = threadIdx.x; k < a.q_stride; k += 256)
        q[k] = k < a.cols && rs.factor != 0.0f ? (int8_t)__builtin_rintf(T::load(x[k]) * rs.factor) : 0;
    if (threadIdx.x == 0)
        a.scale[row] = rs.scale;
}

int launch_quantize(const QuantizeArgs &a, hipStream_t s)
{
    const dim3 grid((uint32_t)a.rows), block(256);
    switch (a.dtype) {
    case RNN_DTYPE_F32: quantize_kernel<F32><<<grid, block, 0, s>>>(a); break;
    case RNN_DTYPE_BF16: quantize_kernel<BF16><<<grid, block, 0, s>>>(a); break;
    default: quantize_kernel<F16><<<grid, block, 0, s>>>(a); break;
    }
    return (int)hipGetLastError();
}

// First form: one output a thread, four products an instruction.
template <class T> __global__ __launch_bounds__(256) void project_kernel(
    rnn_quant_desc d, const int8_t *x, int64_t x_stride, const float *x_scale, const int8_t *w,
    const float *w_scale, const float *bias, void *y)
{
    const int64_t o = (int64_t)blockIdx.x * 64 + threadIdx.x % 64;
    const int64_t i = (int64_t)blockIdx.y * 4 + threadIdx.x / 64;
    if (o >= d.outs || i >= d.rows)
        return;
    const int32_t *xr = (const int32_t *)(x + i * x_stride);
    const int32_t *wr = (const int32_t *)(w + o * d.w_stride);
    int32_t sum = 0;
    const int64_t words = (d.cols + 3) / 4;        // x is zero past cols
    for (int64_t k = 0; k < words; ++k)
        sum = __builtin_amdgcn_sdot4(xr[k], wr[k], sum, false);
    float v = (float)sum * (x_scale[i] * w_scale[o]);
    if (bias)
        v += bias[o];
    ((typename T::raw *)y)[i * d.y_stride + o] = T::store(v);
}

static int64_t pitch(int64_t cols) { return (cols + 127) / 128 * 128; }

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t project_workspace(const rnn_quant_desc &d)
{
    if (d.x_dtype == RNN_DTYPE_I8)
        return 0;
    return up256((size_t)d.rows * pitch(d.cols)) + up256((size_t)d.rows * 4);
}

int launch_project(const ProjectArgs &a, hipStream_t s)
{
    const int8_t *x = (const int8_t *)a.x;
    const float *x_scale = a.x_scale;
    int64_t x_stride = a.d.x_stride;
    if (a.d.x_dtype != RNN_DTYPE_I8) {
        QuantizeArgs q{};
        q.rows = a.d.rows;
        q.cols = a.d.cols;
        q.x_stride = a.d.x_stride;
        q.q_stride = pitch(a.d.cols);
        q.dtype = a.d.x_dtype;
        q.x = a.x;
        q.q = (int8_t *)a.workspace;
        q.scale = (float *)((char *)a.workspace + up256((size_t)q.rows * q.q_stride));
        const int rc = launch_quantize(q, s);
        if (rc)
            return rc;
        x = q.q;
        x_scale = q.scale;
        x_stride = q.q_stride;
    }
    const dim3 grid((uint32_t)((a.d.outs + 63) / 64), (uint32_t)((a.d.rows + 3) / 4)), block(256);
    switch (a.d.y_dtype) {
    case RNN_DTYPE_F32:
        project_kernel<F32><<<grid, block, 0, s>>>(a.d, x, x_stride, x_scale, a.w, a.w_scale, a.bias, a.y);
        break;
    case RNN_DTYPE_BF16:
        project_kernel<BF16><<<grid, block, 0, s>>>(a.d, x, x_stride, x_scale, a.w, a.w_scale, a.bias, a.y);
        break;
    default:
        project_kernel<F16><<<grid, block, 0, s>>>(a.d, x, x_stride, x_scale, a.w, a.w_scale, a.bias, a.y);
        break;
    }
    return (int)hipGetLastError();
}

}  // namespace rnnamd
