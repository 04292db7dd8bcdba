// lm_reorder.hip -- rows of many state tensors in the order of a selection.
//
//   new[o, b, j] = old[o, b, parents[b, j]]
//
// Bound by HBM: each row that is wanted read once, each new one written once.  A
// thread takes 16 bytes (of what is left of a row, one) of all of a request's
// rows, so that in place everything is read before anything is written, and only
// rows that change are touched.  One launch takes up to kReorderItems tensors.
// 1.1 GB of states of 32 rows out of place 165 us, 6.7 TB/s (rows that several take come
// from the caches); 0.5 MB 3.2 us, a launch and two trips to memory, one after another.
#include "lm_common.h"

namespace rnnamd {

// Threads that an item's rows take for each request: whole 16-byte pieces, then bytes.
static __host__ __device__ __forceinline__ uint64_t columns_of(int64_t inner)
{
    return (uint64_t)inner / 16 + (uint64_t)inner % 16;
}

// (a row may begin at any byte; vector elements, since an array of structs does not
// stay in registers)
typedef uint32_t Piece16 __attribute__((ext_vector_type(4), aligned(1)));

// AT rows of a request at a time; in place: all of them.
template <int AT, bool IN_PLACE> __global__ __launch_bounds__(256) void reorder_kernel(ReorderArgs a)
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
    const bool in_place = IN_PLACE && it.in == it.out;
    const int keep = (int)a.keep, beams = (int)a.beams;
    auto rows = [&](auto piece, int64_t at) {
        using Piece = decltype(piece);
        for (int base = 0; base < keep; base += AT) {
            // (all parents, then all rows: a wait each)
            int from[AT];
            Piece v[AT];
#pragma unroll
            for (int j = 0; j < AT; ++j) {
                const int p = parents[base + j < keep ? base + j : keep - 1];
                from[j] = p < 0 ? 0 : p < beams ? p : beams - 1;
            }
#pragma unroll
            for (int j = 0; j < AT; ++j)
                // (past the last row the last one again, which the cache holds)
                if (!(in_place && (base + j >= keep || from[j] == j)))
                    v[j] = *(const Piece *)(in + from[j] * inner + at);
#pragma unroll
            for (int j = 0; j < AT; ++j)
                if (base + j < keep && !(in_place && from[j] == j))
                    *(Piece *)(out + (base + j) * inner + at) = v[j];
        }
    };
    if (column < pieces)
        rows(Piece16{}, 16 * (int64_t)column);
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
    // Out of place 4 rows at a time, or 8: 32 rows 90 us against 93 with 4 at a time, 2 rows
    // 38 against 46 with 8, 5 rows 48 against 58 with 16.  In place everything is read
    // before anything is written.
    if (!in_place) {
        if (a.keep <= 4)
            reorder_kernel<4, false><<<grid, block, 0, s>>>(a);
        else
            reorder_kernel<8, false><<<grid, block, 0, s>>>(a);
    } else if (a.keep <= 4) {
        reorder_kernel<4, true><<<grid, block, 0, s>>>(a);
    } else if (a.keep <= 8) {
        reorder_kernel<8, true><<<grid, block, 0, s>>>(a);
    } else if (a.keep <= 16) {
        reorder_kernel<16, true><<<grid, block, 0, s>>>(a);
    } else if (a.keep <= 32) {
        reorder_kernel<32, true><<<grid, block, 0, s>>>(a);
    } else {
        reorder_kernel<RNN_REORDER_MAX_BEAMS, true><<<grid, block, 0, s>>>(a);
    }
    return (int)hipGetLastError();
}

}  // namespace rnnamd
