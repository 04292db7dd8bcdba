// lm_scores.hip -- log probability of a given token, entropy, rank and the
// most likely alternatives of each row of logits.
//
// First form: a workgroup a row; one pass for the maximum, one for the sums
// and the rank, and one for each alternative.
#include "lm_common.h"

namespace rnnamd {

// The order of the entries: by value, larger first (NaN before all, -0 equal
// to +0), then by index, lower first -- as one number, larger first.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t index)
{
    uint32_t u = __float_as_uint(v + 0.0f);
    u = v != v ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)u << 32) | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v)
{
    for (int m = 32; m > 0; m /= 2) {
        const uint64_t o = __shfl_xor((unsigned long long)v, m, 64);
        v = o > v ? o : v;
    }
    return v;
}

template <class T> __global__ __launch_bounds__(256) void scores_kernel(ScoresArgs a)
{
    using raw = typename T::raw;
    __shared__ uint64_t keys[4];
    __shared__ float sums[2][4];
    __shared__ uint32_t counts[4];
    const int64_t row = blockIdx.x;
    const uint32_t V = (uint32_t)a.d.vocab;
    const raw *x = (const raw *)a.logits + row * a.d.logits_stride;
    const int wave = threadIdx.x / 64;
    int64_t token = -1;
    if (a.tokens)
        token = a.d.token_bytes == 8 ? ((const int64_t *)a.tokens)[row] : ((const int32_t *)a.tokens)[row];
    const bool known = token >= 0 && token < (int64_t)V;
    const float mine = known ? T::load(x[token]) : 0.0f;
    const uint64_t mine_key = known ? order_key(mine, (uint32_t)token) : ~0ull;

    // the largest entry below `below` in the order, over the workgroup
    auto largest = [&](uint64_t below) {
        uint64_t best = 0;
        for (uint32_t v = threadIdx.x; v < V; v += 256) {
            const uint64_t k = order_key(T::load(x[v]), v);
            if (k < below && k > best)
                best = k;
        }
        best = wave_max(best);
        __syncthreads();
        if (threadIdx.x % 64 == 0)
            keys[wave] = best;
        __syncthreads();
        for (int i = 0; i < 4; ++i)
            best = keys[i] > best ? keys[i] : best;
        return best;
    };
    uint64_t key = largest(~0ull);
    const float most = T::load(x[0xFFFFFFFFu - (uint32_t)key]);
    float sum = 0.0f, cross = 0.0f;
    uint32_t before = 0;
    for (uint32_t v = threadIdx.x; v < V; v += 256) {
        const float xv = T::load(x[v]);
        const float e = __builtin_amdgcn_exp2f((xv - most) * kLog2e);
        sum += e;
        cross += e == 0.0f ? 0.0f : e * (xv - most);
        before += order_key(xv, v) > mine_key;
    }
    for (int m = 32; m > 0; m /= 2) {
        sum += __shfl_xor(sum, m, 64);
        cross += __shfl_xor(cross, m, 64);
        before += __shfl_xor(before, m, 64);
    }
    if (threadIdx.x % 64 == 0) {
        sums[0][wave] = sum;
        sums[1][wave] = cross;
        counts[wave] = before;
    }
    __syncthreads();
    sum = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
    cross = sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
    before = counts[0] + counts[1] + counts[2] + counts[3];
    const float lse = __builtin_amdgcn_logf(sum) * kLn2;
    if (threadIdx.x == 0) {
        if (a.logprob)
            a.logprob[row] = known ? (mine - most) - lse : __uint_as_float(0x7FC00000u);
        if (a.entropy)
            a.entropy[row] = lse - cross / sum;
        if (a.rank)
            a.rank[row] = known ? (int32_t)before : -1;
    }
    for (int32_t j = 0; j < a.d.top; ++j) {
        const bool any = j < (int64_t)V;
        if (any && j > 0)
            key = largest(key);
        if (threadIdx.x == 0) {
            const uint32_t at = 0xFFFFFFFFu - (uint32_t)key;
            if (a.top_logprobs)
                a.top_logprobs[row * a.d.top + j] =
                    any ? (T::load(x[at]) - most) - lse : -__builtin_inff();
            if (a.top_ids)
                a.top_ids[row * a.d.top + j] = any ? (int32_t)at : -1;
        }
    }
}

size_t scores_workspace(const rnn_scores_desc &) { return 0; }

int launch_scores(const ScoresArgs &a, hipStream_t s)
{
    const dim3 grid((uint32_t)a.d.rows), block(256);
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: scores_kernel<F32><<<grid, block, 0, s>>>(a); break;
    case RNN_DTYPE_BF16: scores_kernel<BF16><<<grid, block, 0, s>>>(a); break;
    default: scores_kernel<F16><<<grid, block, 0, s>>>(a); break;
    }
    return (int)hipGetLastError();
}

}  // namespace rnnamd
