// lm_reorder.hip -- rows of many state tensors in the order of a selection.
//
//   new[o, b, j] = old[o, b, parents[b, j]]
//
// Bound by HBM: each row that is wanted read once, each new one written once.  A
// thread takes 16 bytes (of what is left of a row, one) of all of a request's
// rows, so that in place everything is read before anything is written, and only
// rows that change are touched.  One launch takes up to kReorderItems tensors.
#include "lm_common.h"

namespace rnnamd {

// Threads that an item's rows take for each request: whole 16-byte pieces, then bytes.
static __host__ __device__ __forceinline__ uint64_t columns_of(int64_t inner)
{
    return (uint64_t)inner / 16 + (uint64_t)inner % 16;
}

// AT rows of a request at a time; in place: all of them.
template <int AT> __global__ __launch_bounds__(256) void reorder_kernel(ReorderArgs a)
{
    int i = 0;
    while (blockIdx.x >= a.first[i + 1])
        ++i;
    const rnn_reorder_item it = a.items[i];
    const uint32_t columns = (uint32_t)columns_of(it.inner_bytes);
    const uint32_t id = (blockIdx.x - a.first[i]) * 256 + threadIdx.x;
    const uint32_t ob = id / columns, column = id % columns;
    if (ob >= it.outer * a.batch)
        return;
    const uint32_t b = ob % (uint32_t)a.batch;
    const int64_t inner = it.inner_bytes, pieces = inner / 16;
    const char *in = (const char *)it.in + (int64_t)ob * a.beams * inner;
    char *out = (char *)it.out + (int64_t)ob * a.keep * inner;
    const int32_t *parents = a.parents + (int64_t)b * a.keep;
    const bool in_place = it.in == it.out;
    const int keep = (int)a.keep, beams = (int)a.beams;
    auto parent = [&](int j) {
        const int p = parents[j];
        return p < 0 ? 0 : p < beams ? p : beams - 1;
    };
    auto rows = [&](auto piece, int64_t at) {
        using Piece = decltype(piece);
        for (int base = 0; base < keep; base += AT) {
            Piece v[AT];
#pragma unroll
            for (int j = 0; j < AT; ++j)
                if (base + j < keep) {
                    const int p = parent(base + j);
                    if (!in_place || p != j)
                        __builtin_memcpy(&v[j], in + p * inner + at, sizeof(Piece));
                }
#pragma unroll
            for (int j = 0; j < AT; ++j)
                if (base + j < keep && (!in_place || parent(base + j) != j))
                    __builtin_memcpy(out + (base + j) * inner + at, &v[j], sizeof(Piece));
        }
    };
    if (column < pieces)
        rows(uint4{}, 16 * (int64_t)column);
    else
        rows(uint8_t{}, 16 * pieces + (column - pieces));
}

int reorder_fits(ReorderArgs &a)
{
    uint64_t blocks = 0;
    for (int i = 0; i < a.count; ++i) {
        const __int128 threads = (__int128)a.items[i].outer * a.batch * columns_of(a.items[i].inner_bytes);
        if (threads > 0xFFFFFFFFu - 256u)
            return (int)hipErrorInvalidConfiguration;
        a.first[i] = (uint32_t)blocks;
        blocks += ((uint64_t)threads + 255) / 256;
        if (!launchable(blocks, 256))
            return (int)hipErrorInvalidConfiguration;
    }
    a.first[a.count] = (uint32_t)blocks;
    return 0;
}

int launch_reorder(ReorderArgs &a, hipStream_t s)
{
    const int rc = reorder_fits(a);
    if (rc)
        return rc;
    bool in_place = false;
    for (int i = 0; i < a.count; ++i)
        in_place |= a.items[i].in == a.items[i].out;
    const dim3 grid(a.first[a.count]), block(256);
    const int64_t at_once = in_place || a.keep < 8 ? a.keep : 8;
    if (at_once <= 4)
        reorder_kernel<4><<<grid, block, 0, s>>>(a);
    else if (at_once <= 8)
        reorder_kernel<8><<<grid, block, 0, s>>>(a);
    else if (at_once <= 16)
        reorder_kernel<16><<<grid, block, 0, s>>>(a);
    else if (at_once <= 32)
        reorder_kernel<32><<<grid, block, 0, s>>>(a);
    else
        reorder_kernel<RNN_REORDER_MAX_BEAMS><<<grid, block, 0, s>>>(a);
    return (int)hipGetLastError();
}

}  // namespace rnnamd
