// lm_project.hip -- matrix product of 8-bit rows.
//
//   y[i,o] = (sum_k qx[i,k] w[o,k]) (x_scale[i] w_scale[o]) + bias[o]
//
// Many rows: bound by the matrix unit (and the clock, which falls under it);
// tiles of x and w go to LDS by direct loads, 32x32x32 products, the scales in
// the epilogue: 8192^3 in 487 us (2.26 POPS), 8192 x 2048 x 8192 in 158 us once the
// clock has settled (up to 190 in the first milliseconds of such work).
// Few rows: bound by reading w once; it goes from memory to the matrix unit's
// registers: 4 x 2048 x 8192 in 7.6 us.
#include <type_traits>
#include <utility>

#include "lm_common.h"

namespace rnnamd {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

struct ProjectGo {
    const int8_t *x, *w;
    const float *x_scale, *w_scale, *bias;
    void *y;
    int64_t x_stride, w_stride, y_stride;
    int32_t rows, outs;
    int32_t k_end;          // columns, rounded up to 16 (the pitch of both sides reaches it)
    int32_t x_end;          // columns of x that count: k_end where it has zeros past the last
};

// The first n (none below 1, all from 16) of 16 columns, zeros behind them.
__device__ __forceinline__ v4i first_columns(v4i v, int n)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = n - 4 * i;
        v[i] &= b >= 4 ? -1 : b > 0 ? (1 << 8 * b) - 1 : 0;
    }
    return v;
}

// ---------------------------------------------------------------------------
// Many rows.  A workgroup has BM tokens x BN outputs, WM x WN waves, or WK of
// them that take a part of the columns each.  A step is 64 columns (of each
// part): a tile row is 64 bytes of LDS, whose 16-byte pieces are
// permuted by the row (piece p of row r holds columns 16 (p xor r/4%4) on), so
// that the sixteen rows that one pass of a 16-byte read takes (lanes 0-3, 12-15,
// 20-23, 24-27, then the others) are in different banks.  The permutation is applied
// to the addresses that the direct loads read from: in LDS they write in order.
// BUFFERS steps have a buffer each (four; three where the columns are divided): the
// loads of BUFFERS - 1 steps are in flight during the products of one, and a wave
// waits for its own part of the next step only (by count), then for the others at
// the step's one barrier.  Operands are read half a step ahead, between the
// products of the half before.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void load_to_lds(const int8_t *p, int8_t *lds)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)p,
                                     (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// Until at most N of the wave's loads are out (they come in order), and none
// of its reads of LDS.
template <int N> __device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// READS reads of LDS (a later half's operands) and LOADS loads (a later step's)
// spread between the products I...: a product takes 4 cycles to issue and runs
// for 32.
template <int READS, int LOADS, int... I>
__device__ __forceinline__ void interleave(std::integer_sequence<int, I...>)
{
    constexpr int N = sizeof...(I);
    ((__builtin_amdgcn_sched_group_barrier(0x008, 1, 0),
      __builtin_amdgcn_sched_group_barrier(0x100, READS * (I + 1) / N - READS * I / N, 0),
      __builtin_amdgcn_sched_group_barrier(0x020, LOADS * (I + 1) / N - LOADS * I / N, 0)),
     ...);
}

template <class T, int BM, int BN, int WM, int WN, int WK, int BUFFERS>
__global__ __launch_bounds__(64 * WM * WN * WK) void project_tiles_kernel(ProjectGo g, uint32_t m_tiles,
                                                                    uint32_t n_tiles)
{
    using raw = typename T::raw;
    constexpr int WAVES = WM * WN * WK, THREADS = 64 * WAVES, KB = 64;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;       // 32 x 32 tiles of a wave
    constexpr int XP = BM * 4 * WK / THREADS, WP = BN * 4 * WK / THREADS;   // pieces a thread loads
    // Epilogue: rows of ON outputs, V of a thread (16 bytes), R rows a pass
    constexpr int ON = TN * 32, OP = ON + 4, V = 16 / sizeof(raw), R = 64 / (ON / V);
    constexpr int ROWS = WK == 1 ? TM * 32 : BM / WK, PASSES = ROWS / R;    // of a wave
    constexpr int BUFFER = WK * (BM + BN) * KB;
    constexpr int SUMS = (WK == 1 ? WAVES * 32 : WK * BM) * OP * 4;
    static_assert(WK == 1 || (WM == 1 && WN == 1), "columns are divided among single waves");
    __shared__ __attribute__((aligned(128))) int8_t lds[BUFFERS * BUFFER > SUMS ? BUFFERS * BUFFER : SUMS];

    // Tiles in bands of 8 tiles of tokens, each XCD (workgroups go to them in
    // turn) a run of adjacent ones: what runs at a time on an XCD shares rows of
    // both sides in its L2.
    const uint32_t total = gridDim.x, xcd = blockIdx.x % 8, q8 = total / 8, r8 = total % 8;
    const uint32_t id = xcd * q8 + (xcd < r8 ? xcd : r8) + blockIdx.x / 8;
    const uint32_t band = id / (8 * n_tiles), in = id % (8 * n_tiles);
    const uint32_t high = m_tiles - band * 8 < 8 ? m_tiles - band * 8 : 8;
    const int row0 = (int)((band * 8 + in % high) * BM), out0 = (int)(in / high * BN);

    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int wk = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;

    // rows past the end repeat the last one; their outputs are not stored
    const int8_t *xp[XP], *wp[WP];
    int kx[XP], kw[WP];
#pragma unroll
    for (int i = 0; i < XP; ++i) {
        const int q = i * THREADS + tid, r = q / 4 % BM;
        const int row = row0 + r < g.rows ? row0 + r : g.rows - 1;
        kx[i] = q / (4 * BM) * KB + (q % 4 ^ (r / 4 & 3)) * 16;
        xp[i] = g.x + (int64_t)row * g.x_stride + kx[i];
    }
#pragma unroll
    for (int i = 0; i < WP; ++i) {
        const int q = i * THREADS + tid, r = q / 4 % BN;
        const int row = out0 + r < g.outs ? out0 + r : g.outs - 1;
        kw[i] = q / (4 * BN) * KB + (q % 4 ^ (r / 4 & 3)) * 16;
        wp[i] = g.w + (int64_t)row * g.w_stride + kw[i];
    }
    auto stage = [&](int k) {
        int8_t *X = lds + k % BUFFERS * BUFFER, *W = X + WK * BM * KB;
#pragma unroll
        for (int i = 0; i < XP; ++i)
            load_to_lds(xp[i] + k * (KB * WK), X + (i * THREADS + wave * 64) * 16);
#pragma unroll
        for (int i = 0; i < WP; ++i)
            load_to_lds(wp[i] + k * (KB * WK), W + (i * THREADS + wave * 64) * 16);
    };

    // the scales of the epilogue's rows and columns, on their way from the start
    const int o = out0 + wn * ON + lane % (ON / V) * V;
    const int row_first = row0 + (WK == 1 ? wm * TM * 32 : wave * ROWS) + lane / (ON / V);
    float ws[V], bs[V] = {}, xs[PASSES];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = o + v < g.outs ? o + v : g.outs - 1;
        ws[v] = g.w_scale[col];
        if (g.bias)
            bs[v] = g.bias[col];
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
        xs[i] = g.x_scale[row_first + i * R < g.rows ? row_first + i * R : g.rows - 1];

    v16i acc[TN][TM];
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int m = 0; m < TM; ++m)
            acc[n][m] = v16i{};
    // Operands of half a step (32 columns), and the products of them.
    struct Half {
        v4i x[TM], w[TN];
    };
    auto fetch = [&](int k, int half, Half &f) {
        const int8_t *X = lds + k % BUFFERS * BUFFER + wk * BM * KB;
        const int8_t *W = lds + k % BUFFERS * BUFFER + WK * BM * KB + wk * BN * KB;
        const int at = ((half * 2 + lane / 32) ^ (lane / 4 & 3)) * 16;
        X += (wm * TM * 32 + lane % 32) * KB + at;
        W += (wn * TN * 32 + lane % 32) * KB + at;
#pragma unroll
        for (int m = 0; m < TM; ++m)
            f.x[m] = *(const v4i *)(X + m * 32 * KB);
#pragma unroll
        for (int n = 0; n < TN; ++n)
            f.w[n] = *(const v4i *)(W + n * 32 * KB);
    };
    auto products = [&](const Half &f) {
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int m = 0; m < TM; ++m)
                acc[n][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[n], f.x[m], acc[n][m], 0, 0, 0);
    };
    using Products = std::make_integer_sequence<int, TM * TN>;

    const int steps = g.x_end / (KB * WK);      // whole ones
#pragma unroll
    for (int k = 0; k < BUFFERS; ++k)
        if (k < steps)
            stage(k);
    // Step k, whose first half (even) has been read.  Before its barrier each wave has
    // read the second half too and waited for that read (lgkmcnt) and for its own
    // loads of step k + 1 (vmcnt; those of the BUFFERS - 2 steps after may be out).
    // So after it step k + 1 is there for all, and nobody reads step k any more, whose
    // buffer step k + BUFFERS gets: fetch(k, 1) has to stay above the wait.
    auto step = [&](int k, Half &even, Half &odd, auto more) {
        constexpr bool MORE = decltype(more)::value;
        fetch(k, 1, odd);
        products(even);
        interleave<TM + TN, 0>(Products{});
        wait_loads<MORE ? (BUFFERS - 2) * (XP + WP) : 0>();
        __builtin_amdgcn_s_barrier();
        if (MORE)
            stage(k + BUFFERS);
        fetch(k + 1, 0, even);
        products(odd);
        if (MORE)
            interleave<TM + TN, XP + WP>(Products{});
        else
            interleave<TM + TN, 0>(Products{});
    };
    if (steps > 0) {
        Half even, odd;
        if (steps >= BUFFERS)
            wait_loads<(BUFFERS - 1) * (XP + WP)>();
        else
            wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        fetch(0, 0, even);
        int k = 0;
        for (; k + BUFFERS < steps; ++k)
            step(k, even, odd, std::true_type{});
        for (; k + 1 < steps; ++k)
            step(k, even, odd, std::false_type{});
        fetch(steps - 1, 1, odd);
        products(even);
        products(odd);
    }
    if (g.x_end % (KB * WK)) {                  // the last columns, zeros behind them
        const int k0 = steps * (KB * WK);
        int8_t *X = lds + steps % BUFFERS * BUFFER, *W = X + WK * BM * KB;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            v4i v = k0 + kx[i] < g.k_end ? *(const v4i *)(xp[i] + k0) : v4i{};
            if (g.x_end < g.k_end)
                v = first_columns(v, g.x_end - k0 - kx[i]);
            *(v4i *)(X + (i * THREADS + tid) * 16) = v;
        }
#pragma unroll
        for (int i = 0; i < WP; ++i)
            *(v4i *)(W + (i * THREADS + tid) * 16) =
                k0 + kw[i] < g.k_end ? *(const v4i *)(wp[i] + k0) : v4i{};
        __syncthreads();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            Half f;
            fetch(steps, half, f);
            products(f);
        }
    }
    __syncthreads();

    // Epilogue.  A lane holds groups of four outputs of one token; through LDS
    // it gets V adjacent outputs of a token, and R rows go out as whole pieces.
    // A wave uses a part of its own, 32 tokens at a time; waves with parts of the
    // columns put down all their sums first, and each adds up some of the rows.
    int *tile = (int *)lds + (WK == 1 ? wave * 32 : wk * BM) * OP;
    auto put_down = [&](int m, int *to) {
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                *(v4i *)(to + lane % 32 * OP + n * 32 + 8 * v + 4 * (lane / 32)) =
                    v4i{acc[n][m][4 * v], acc[n][m][4 * v + 1], acc[n][m][4 * v + 2], acc[n][m][4 * v + 3]};
    };
    auto pass = [&](int i, const int *from) {
        v4i sum[V / 4];
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            sum[q] = *(const v4i *)(from + 4 * q);
#pragma unroll
            for (int part = 1; part < WK; ++part)
                sum[q] += *(const v4i *)(from + part * BM * OP + 4 * q);
        }
        const int row = row_first + i * R;
        if (row >= g.rows)
            return;
        Pack<T, V> out;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f = (float)sum[v / 4][v % 4] * (xs[i] * ws[v]);
            if (g.bias)
                f += bs[v];
            out.v[v] = T::store(f);
        }
        raw *y = (raw *)g.y + (int64_t)row * g.y_stride + o;
        if (o + V <= g.outs) {
            store_pack<T, V>(y, out);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (o + v < g.outs)
                    y[v] = out.v[v];
        }
    };
    const int at = lane / (ON / V) * OP + lane % (ON / V) * V;
    if constexpr (WK == 1) {
#pragma unroll
        for (int m = 0; m < TM; ++m) {
            put_down(m, tile);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 32 / R; ++i)
                pass(m * (32 / R) + i, tile + i * R * OP + at);
            __builtin_amdgcn_wave_barrier();
        }
    } else {
#pragma unroll
        for (int m = 0; m < TM; ++m)
            put_down(m, tile + m * 32 * OP);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PASSES; ++i)
            pass(i, (const int *)lds + (wave * ROWS + i * R) * OP + at);
    }
}

// ---------------------------------------------------------------------------
// Few rows (up to 16, and at least a column).  A workgroup has 16 outputs; its four waves take steps
// of 128 columns in turn and add their sums in LDS.  A load takes 64 bytes of
// 16 weight rows, straight into the operands of 16x16x64 products.  With FROM (the rows' type) x is rounded in the
// call: each workgroup does it for itself, into LDS, while its first weights
// are on their way; that is less than a launch for few elements.
// ---------------------------------------------------------------------------

constexpr int kFewRows = 16;
constexpr int kFusedElements = 16384;      // most elements of x to round inside

struct NoSource {};

template <class T, class FROM>
__global__ __launch_bounds__(256) void project_rows_kernel(ProjectGo g, const void *x_source,
                                                          int64_t source_stride, int32_t cols)
{
    constexpr bool FUSED = !std::is_same<FROM, NoSource>::value;
    constexpr int AHEAD = 2;                     // steps of a group; two are in flight
    extern __shared__ __attribute__((aligned(16))) int8_t q_lds[];   // FUSED: rows of pitch, then scales
    __shared__ __attribute__((aligned(16))) int sums[3][256];
    __shared__ uint32_t row_max[16];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int out0 = blockIdx.x * 16;
    const int steps = (g.k_end + 127) / 128;
    const int pitch = steps * 128 + 16;
    float *q_scale = (float *)(q_lds + g.rows * pitch);

    // a thread's packs of 8 elements of x, 256 apart, row after row
    constexpr int KEEP = FUSED ? kFusedElements / 8 / 256 : 1;
    const int row_packs = steps * 16;
    typedef typename std::conditional<FUSED, FROM, BF16>::type X;
    Pack<X, 8> keep[KEEP];
    // (a pack's number and row_packs are below 2^12: the quotient is right)
    const float of_row = 1.0f / (float)row_packs;
    auto row_of = [&](int j) { return (int)(((float)(threadIdx.x + 256 * j) + 0.5f) * of_row); };
    if constexpr (FUSED) {
        if (threadIdx.x < 16)
            row_max[threadIdx.x] = 0;
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            const int r = row_of(j), k = ((int)threadIdx.x + 256 * j - r * row_packs) * 8;
            const typename X::raw *x = (const typename X::raw *)x_source + r * source_stride + k;
            keep[j] = Pack<X, 8>{};
            if (r < g.rows) {
                if (k + 8 <= cols) {
                    keep[j] = load_pack<X, 8>(x);
                } else {
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        if (k + v < cols)
                            keep[j].v[v] = x[v];
                }
            }
        }
    }

    const int wrow = out0 + lane % 16 < g.outs ? out0 + lane % 16 : g.outs - 1;
    const int xrow = lane % 16 < g.rows ? lane % 16 : g.rows - 1;
    const int8_t *w = g.w + (int64_t)wrow * g.w_stride;
    const int8_t *x = FUSED ? q_lds + xrow * pitch : g.x + (int64_t)xrow * g.x_stride;
    // Past the last columns the last ones are loaded again (no load depends on a
    // condition: it would be waited for on the spot); x is zero there.
    auto piece = [&](const int8_t *p, int k) {
        return *(const v4i *)(p + (k < g.k_end ? k : g.k_end - 16));
    };
    struct Group {                      // AHEAD steps of the wave, from its step `s`
        v4i w[AHEAD][2], x[AHEAD][2];
    };
    auto fetch = [&](int s, Group &f) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (s + 4 * i) * 128 + lane / 16 * 16 + 64 * h;
                f.w[i][h] = piece(w, k);
                if (!FUSED)
                    f.x[i][h] = piece(x, k);
            }
    };
    Group first, second;
    fetch(wave, first);

    if constexpr (FUSED) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            const int r = row_of(j);
            uint32_t most = pack_max<X, 8>(keep[j], 0);
            if (256 * j >= g.rows * row_packs)
                break;
            // one addition to LDS for a wave that is in one row
            if (__builtin_amdgcn_readfirstlane(r) == __builtin_amdgcn_readlane(r, 63)) {
                most = wave_max(most);
                if (lane == 0 && r < g.rows)
                    atomicMax(&row_max[r], most);
            } else if (r < g.rows) {
                atomicMax(&row_max[r], most);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            const int r = row_of(j), k = ((int)threadIdx.x + 256 * j - r * row_packs) * 8;
            if (r >= g.rows)
                break;
            const uint32_t most = row_max[r];
            const RowScale rs = row_scale(__uint_as_float(most), most < kInfBits);
            *(uint2 *)(q_lds + r * pitch + k) = pack_8bit<X>(keep[j], rs.factor);
            if (k == 0)
                q_scale[r] = rs.scale;
        }
        __syncthreads();
    }

    v4i acc = v4i{};
    auto products = [&](int s, const Group &f) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (s + 4 * i) * 128 + lane / 16 * 16 + 64 * h;
                v4i b = FUSED ? *(const v4i *)(x + (s + 4 * i < steps ? k : 0)) : f.x[i][h];
                if (FUSED ? s + 4 * i >= steps : (s + 4 * i + 1) * 128 > g.x_end)
                    b = first_columns(b, g.x_end - k);
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[i][h], b, acc, 0, 0, 0);
            }
    };
    for (int s = wave;; s += 8 * AHEAD) {
        if (s + 4 * AHEAD >= steps) {
            products(s, first);
            break;
        }
        fetch(s + 4 * AHEAD, second);
        products(s, first);
        if (s + 8 * AHEAD >= steps) {
            products(s + 4 * AHEAD, second);
            break;
        }
        fetch(s + 8 * AHEAD, first);
        products(s + 4 * AHEAD, second);
    }
    // a lane has outputs 4 (lane / 16) to + 3 of row lane % 16
    if (wave > 0)
        *(v4i *)&sums[wave - 1][lane * 4] = acc;
    __syncthreads();
    const int row = lane % 16, o = out0 + lane / 16 * 4;
    if (wave > 0 || row >= g.rows)
        return;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        acc += *(const v4i *)&sums[i][lane * 4];
    const float xs = FUSED ? q_scale[row] : g.x_scale[row];
    typename T::raw *y = (typename T::raw *)g.y + (int64_t)row * g.y_stride + o;
    Pack<T, 4> out;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int oo = o + v < g.outs ? o + v : g.outs - 1;
        float f = (float)acc[v] * (xs * g.w_scale[oo]);
        if (g.bias)
            f += g.bias[oo];
        out.v[v] = T::store(f);
    }
    if (o + 4 <= g.outs) {
        store_pack<T, 4>(y, out);
    } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (o + v < g.outs)
                y[v] = out.v[v];
    }
}

// ---------------------------------------------------------------------------

static int64_t pitch(int64_t cols) { return (cols + 127) / 128 * 128; }
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

static bool fused(const rnn_quant_desc &d)
{
    return d.x_dtype != RNN_DTYPE_I8 && d.cols > 0 && d.rows <= kFewRows && d.rows * pitch(d.cols) <= kFusedElements;
}

size_t project_workspace(const rnn_quant_desc &d)
{
    if (d.x_dtype == RNN_DTYPE_I8 || fused(d))
        return 0;
    return up256((size_t)d.rows * pitch(d.cols)) + up256((size_t)d.rows * 4);
}

template <class T, int BM, int BN, int WM, int WN, int WK, int BUFFERS>
static void tiles_go(const ProjectGo &g, hipStream_t s)
{
    const uint32_t m = (uint32_t)((g.rows + (int64_t)BM - 1) / BM);
    const uint32_t n = (uint32_t)((g.outs + (int64_t)BN - 1) / BN);
    project_tiles_kernel<T, BM, BN, WM, WN, WK, BUFFERS>
        <<<dim3(m * n), dim3(64 * WM * WN * WK), 0, s>>>(g, m, n);
}

static int64_t tiles(const ProjectGo &g, int64_t bm, int64_t bn)
{
    return (g.rows + bm - 1) / bm * ((g.outs + bn - 1) / bn);
}

// Whether project_rows_kernel takes it.  Each of its workgroups reads all of x:
// with 64 MiB of weights or more the tiles are faster for rows that are 8-bit
// already, or that another launch rounds (16 rows x 8192 columns x 16384 outputs:
// 22 us against 32; 8192 outputs of 2048 columns: 9.0 against 8.8 and no launch to
// round).
static bool by_rows(const ProjectGo &g, const rnn_quant_desc &d)
{
    const bool heavy = (int64_t)g.outs * g.k_end >= (int64_t)64 << 20 && tiles(g, 64, 64) >= 192;
    return fused(d) || (g.rows <= kFewRows && d.cols > 0 && !heavy);
}

template <class T> static int project_go(const ProjectGo &g, const ProjectArgs &a, hipStream_t s)
{
    const dim3 few((uint32_t)((g.outs + (int64_t)15) / 16));
    const int32_t cols = (int32_t)a.d.cols;
    if (fused(a.d)) {
        const size_t lds = (size_t)g.rows * (pitch(cols) + 16) + g.rows * 4;
        switch (a.d.x_dtype) {
        case RNN_DTYPE_F32:
            project_rows_kernel<T, F32><<<few, 256, lds, s>>>(g, a.x, a.d.x_stride, cols);
            break;
        case RNN_DTYPE_BF16:
            project_rows_kernel<T, BF16><<<few, 256, lds, s>>>(g, a.x, a.d.x_stride, cols);
            break;
        default:
            project_rows_kernel<T, F16><<<few, 256, lds, s>>>(g, a.x, a.d.x_stride, cols);
            break;
        }
        return (int)hipGetLastError();
    }
    if (by_rows(g, a.d)) {
        project_rows_kernel<T, NoSource><<<few, 256, 0, s>>>(g, nullptr, 0, cols);
        return (int)hipGetLastError();
    }
    // The largest tiles that give most of the 256 compute units one; oblong ones
    // only where they are all there at once (1024 x 8192 x 8192: 256 of 256 x 128 78 us,
    // 128 x 128 85 us; 256 x 8192 x 8192: 256 of 128 x 64 34 us, 64 x 64 39 us; but
    // 3388 x 896 x 2838: 322 of 256 x 128 27 us, 128 x 128 22 us).  The smallest
    // ones, if they are all there at once, with the columns divided among the
    // waves, a quarter of the steps (2238 rows x 6607 columns x 68 outputs: 14.7
    // us against 17.5; with more tiles than that its memory of LDS, one workgroup
    // a unit, costs more: 777 x 1500 x 2101 13.2 against 10.6).
    auto one_each = [&](int64_t n) { return n >= 192 && n <= 256; };
    if (tiles(g, 256, 256) >= 192)
        tiles_go<T, 256, 256, 2, 4, 1, 4>(g, s);
    else if (one_each(tiles(g, 256, 128)))
        tiles_go<T, 256, 128, 4, 2, 1, 4>(g, s);
    else if (tiles(g, 128, 128) >= 192)
        tiles_go<T, 128, 128, 2, 2, 1, 4>(g, s);
    else if (one_each(tiles(g, 128, 64)))
        tiles_go<T, 128, 64, 2, 2, 1, 4>(g, s);
    else if (tiles(g, 64, 64) > 256)
        tiles_go<T, 64, 64, 2, 2, 1, 4>(g, s);
    else
        tiles_go<T, 64, 64, 1, 1, 4, 3>(g, s);
    return (int)hipGetLastError();
}

int launch_project(const ProjectArgs &a, hipStream_t s)
{
    ProjectGo g{};
    g.x = (const int8_t *)a.x;
    g.w = a.w;
    g.x_scale = a.x_scale;
    g.w_scale = a.w_scale;
    g.bias = a.bias;
    g.y = a.y;
    g.x_stride = a.d.x_stride;
    g.w_stride = a.d.w_stride;
    g.y_stride = a.d.y_stride;
    g.rows = (int32_t)a.d.rows;
    g.outs = (int32_t)a.d.outs;
    g.k_end = (int32_t)((a.d.cols + 15) / 16 * 16);
    g.x_end = a.d.x_dtype == RNN_DTYPE_I8 ? (int32_t)a.d.cols : g.k_end;
    // (tiles smaller than the largest are a few thousand at most)
    if (!(by_rows(g, a.d) ? launchable(((uint64_t)g.outs + 15) / 16, 256)
                          : launchable((uint64_t)tiles(g, 256, 256), 512)))
        return (int)hipErrorInvalidConfiguration;
    if (a.d.x_dtype != RNN_DTYPE_I8 && !fused(a.d)) {
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
        g.x = q.q;
        g.x_scale = q.scale;
        g.x_stride = q.q_stride;
    }
    switch (a.d.y_dtype) {
    case RNN_DTYPE_F32: return project_go<F32>(g, a, s);
    case RNN_DTYPE_BF16: return project_go<BF16>(g, a, s);
    default: return project_go<F16>(g, a, s);
    }
}

}  // namespace rnnamd
