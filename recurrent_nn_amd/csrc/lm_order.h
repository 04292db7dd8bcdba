// lm_order.h -- the order of logits by value and index, and the first of them:
// shared by the token scores and the selection over beams.
#pragma once

#include "lm_common.h"

namespace rnnamd {

// The order of the entries: by value, larger first (NaN before all, -0 equal
// to +0), then by index, lower first -- as one number, larger first, never 0.
__device__ __forceinline__ uint32_t value_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return v != v ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t u)
{
    return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint64_t order_key(float v, uint32_t index)
{
    return ((uint64_t)value_key(v) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float key_value(uint64_t key) { return value_of((uint32_t)(key >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// The best `top` of the keys given to it, in order.  All threads of a
// workgroup of 256 call its functions together.
constexpr int kList = 512;
struct Best {
    uint64_t *list;         // [kList] of LDS
    uint64_t *sorted;       // [RNN_SCORES_MAX_TOP]
    uint32_t *count;
    int top;
    uint64_t bound;         // what no longer counts: the last of `top` kept keys
    uint32_t kept;          // in order
    uint32_t settled;       // of the list that stay if what is offered next does not fit

    __device__ void begin(uint64_t *l, uint64_t *s, uint32_t *c, int k)
    {
        list = l, sorted = s, count = c, top = k, bound = 0, kept = settled = 0;
        if (threadIdx.x == 0)
            *count = 0;
        __syncthreads();
    }
    __device__ __forceinline__ void offer(uint64_t key, bool on)
    {
        if (on && key > bound) {
            const uint32_t at = atomicAdd(count, 1u);
            if (at < kList)
                list[at] = key;
        }
    }
    // N keys at once, those of `wanted` (a bit each): one addition to the count.
    template <int N> __device__ __forceinline__ void offer(const uint64_t (&key)[N], uint32_t wanted)
    {
#pragma unroll
        for (int v = 0; v < N; ++v)
            wanted &= ~((uint32_t)!(key[v] > bound) << v);
        if (wanted == 0)
            return;
        uint32_t at = atomicAdd(count, (uint32_t)__popc(wanted));
#pragma unroll
        for (int v = 0; v < N; ++v)
            if (wanted >> v & 1) {
                if (at < kList)
                    list[at] = key[v];
                ++at;
            }
    }
    // How many the list has been offered, kept ones among them.  The caller either
    // settles them, or gives up on what came since the last time with forget().
    __device__ __forceinline__ uint32_t offered()
    {
        __syncthreads();
        const uint32_t n = *count;
        __syncthreads();
        return n;
    }
    __device__ __forceinline__ void settle(uint32_t n) { settled = n; }
    __device__ void forget()
    {
        if (threadIdx.x == 0)
            *count = settled;
        __syncthreads();
    }
    // Each key's place is the number of larger ones.
    __device__ void order(uint32_t n)
    {
        for (uint32_t i = threadIdx.x; i < n; i += 256) {
            const uint64_t key = list[i];
            uint32_t place = 0;
#pragma unroll 8
            for (uint32_t j = 0; j < n; ++j)
                place += list[j] > key;
            if (place < (uint32_t)top)
                sorted[place] = key;
        }
        __syncthreads();
        kept = settled = n < (uint32_t)top ? n : (uint32_t)top;
        if (threadIdx.x < kept)
            list[threadIdx.x] = sorted[threadIdx.x];
        if (threadIdx.x == 0)
            *count = kept;
        if (n >= (uint32_t)top)
            bound = sorted[top - 1];
        __syncthreads();
    }
};

template <class T> __device__ __forceinline__ Pack<T, 8> logits_pack(const typename T::raw *x,
                                                                    uint32_t i, uint32_t V)
{
    if (8 * i + 8 <= V)
        return load_pack<T, 8>(x + 8 * (int64_t)i);
    Pack<T, 8> p;
#pragma unroll
    for (uint32_t v = 0; v < 8; ++v)
        p.v[v] = 8 * i + v < V ? x[8 * (int64_t)i + v] : T::store(-__builtin_inff());
    return p;
}

}  // namespace rnnamd
