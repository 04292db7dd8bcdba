// lm_delta_chunk.hip -- gated delta rule in chunks of 64 steps, on the matrix
// cores.
//
// With the state S before a chunk, G_i the sum of the chunk's log decays up to
// step i, and L_ij = b_i e^(G_i - G_j) k_i . k_j for j < i, the corrections of all
// the chunk's steps solve one triangular system, and the rest are products:
//     (1 + L) U = b (V - e^G K S)
//     O = scale (e^G Q S + P' U),   P'_ij = e^(G_i - G_j) q_i . k_j for j <= i
//     S = e^(G_63) S + K^T (e^(G_63 - G) U)
// Only products of decays forward in time occur, so nothing overflows that the
// steps themselves would not, and differences of G are taken in twice the bits.
//
// A first kernel, a workgroup for each chunk and head, makes what does not depend
// on S: T = (1 + L)^-1 b, P = scale P', the decays, and K transposed.  The inverse
// is by forward substitution (16 x 16 blocks, and blocks below them from those):
// powers of L, which double the steps at once, exceed it by orders of magnitude
// where keys are alike.  A second kernel walks along the chunks, a workgroup for
// each head and 16 columns of its state, which never leaves the registers but as
// an operand.
//
// Matrix cores take bfloat16; what has more bits is split into planes that
// add up to it: float32 (S, R, U, T) into three, exactly, and float16 into two.  Of
// the products of planes those of the first 24 bits are taken (16 for outputs in
// 16 bits), so sums are those of float32.  Norms, decays and rates are factors of
// rows of the products, so bfloat16 keys and queries are operands as they are.
//
// A product's result is the next one's operand without a transposition: the
// matrix cores give a lane four rows of a column and take eight from it, and the
// order in which rows are summed over is free.  Row i of a chunk is row m of tile
// w with i = 32 (w / 2) + 8 (m / 4) + 4 (w % 2) + m % 4, so that the tiles 2 p and
// 2 p + 1 together are an operand of 32 rows; likewise rows of the state.
//
// One row of 8192 steps, 32 heads over 16 key heads, 128 x 128, bf16: 76 us and 245 us.
// The first kernel's chunks are independent; their chains (the forward substitution, LDS
// between the steps) and 0.23 GB that it writes bound it, the matrix cores are busy 7% of
// it.  The second is a chain along the chunks, 1.9 us each on every compute unit: 1.2 us of
// it are the products and LDS between them (157 us in all with every load taken out), the
// rest is the reading of 88 KB of operands a chunk by each of a head's eight workgroups
// from the L2, 3.2 GB at 13 TB/s.  The matrix cores are busy 16%.
#include <type_traits>

#include "lm_delta.h"

namespace rnnamd {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kChunk = 64;
constexpr int kFragment = 1024;         // bytes of an operand of 16 x 32: 16 for each lane
constexpr int kLower = 6;               // operands of a 64 x 64 lower triangle

template <class T> constexpr int kPlanes = 1;
template <> constexpr int kPlanes<F16> = 2;
template <> constexpr int kPlanes<F32> = 3;
// The last power of 2^-8 whose products count for outputs of this type.
template <class T> constexpr int kOutLast = std::is_same<T, F32>::value ? 2 : 1;

__device__ __forceinline__ v4f mfma(v8b a, v8b b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma(float a, float b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// N values (an even number) as planes: P bfloat16 values that add up to each, the
// first the nearest, each other the nearest to what is left.  Two values a
// conversion; the last plane's remainder is not taken.
template <int P, int N> struct Planes {
    uint32_t pair[P][N / 2];
    __device__ __forceinline__ explicit Planes(const float (&x)[N])
    {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            float lo = x[2 * j], hi = x[2 * j + 1];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                typedef __bf16 v2b __attribute__((ext_vector_type(2)));
                typedef float v2f __attribute__((ext_vector_type(2)));
                const uint32_t both = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2b));
                pair[p][j] = both;
                if (p + 1 < P) {
                    lo -= __uint_as_float(both << 16);
                    hi -= __uint_as_float(both & 0xFFFF0000u);
                }
            }
        }
    }
    __device__ __forceinline__ void put(int p, void *to) const { __builtin_memcpy(to, pair[p], 2 * N); }
};

// Row m of tile w of a chunk (or of a state), and the place of a row in that order.
__device__ __forceinline__ int row_of(int w, int m) { return 32 * (w / 2) + 8 * (m / 4) + 4 * (w % 2) + m % 4; }
__device__ __forceinline__ int place_of(int i) { return 16 * (2 * (i / 32) + i % 8 / 4) + 4 * (i % 32 / 8) + i % 4; }
// The operands of a lower triangle: tiles 0 and 1 have one, 2 and 3 two.
__device__ __forceinline__ int lower_of(int w, int p) { return w < 2 ? w : 2 * w - 2 + p; }

// What one pair of launches does.
struct DeltaSpan {
    uint32_t first, count;              // chunks
    char *t, *p, *vec;                  // for each head and chunk: T, P, factors of rows
    char *kt, *packed;                  // for each key head and chunk: K transposed; K and Q
    const float *from;                  // states before
    float *to;                          // and after
};
constexpr int kVec = 256;               // floats: e^G |k|, scale e^G |q|, e^(G_63 - G) |k|, e^G_63

template <class T, int KB> struct DeltaSizes {
    static constexpr size_t t = 3 * kLower * kFragment;
    static constexpr size_t p = (kOutLast<T> + 1) * kLower * kFragment;
    static constexpr size_t vec = kVec * sizeof(float);
    static constexpr size_t kt = (size_t)kPlanes<T> * 4 * KB * kFragment;
};

// The workgroup's head of the batch and its place in that; heads go round the
// XCDs, so that what shares keys and chunks shares an L2.
struct Place {
    uint32_t bh, at;
};
__device__ __forceinline__ Place place_in(uint32_t each)
{
    const uint32_t i = blockIdx.x / 8;
    return {i / each * 8 + blockIdx.x % 8, i % each};
}

template <class T, int KB, bool DIRECT, bool WHOLE>
__global__ __launch_bounds__(256) void delta_prepare_kernel(DeltaArgs a, DeltaSpan sp)
{
    using raw = typename T::raw;
    constexpr int KP = kPlanes<T>, PP = kOutLast<T> + 1, LDK = 32 * KB + 8, LDT = 68;
    using Sizes = DeltaSizes<T, KB>;
    __shared__ __attribute__((aligned(16))) __bf16 keys[KP][kChunk][LDK];
    // L transposed above the diagonal, (1 + L)^-1 on it and below
    __shared__ __attribute__((aligned(16))) float M[kChunk][LDT];
    __shared__ float2 G2[kChunk];               // sums of log2 decays, and what float32 leaves of them
    __shared__ __attribute__((aligned(16))) float rates[kChunk], rk[kChunk], rq[kChunk];
    const int tid = threadIdx.x, lane = tid % 64, w = __builtin_amdgcn_readfirstlane(tid / 64);
    const int n16 = lane % 16, g = lane / 16;
    const Place pl = place_in(sp.count);
    const uint32_t heads = (uint32_t)a.d.heads;
    const int64_t b = pl.bh / heads, head = pl.bh % heads;
    if (b >= a.d.batch)
        return;
    const int n = delta_steps(a, b), start = (int)((sp.first + pl.at) * kChunk);
    if (start >= n)
        return;
    const int here = n - start < kChunk ? n - start : kChunk;
    const int64_t each = a.d.heads / a.d.key_heads, key_head = head / each;
    const int dk = (int)a.d.key_dim;
    const size_t unit = (size_t)pl.bh * sp.count + pl.at;
    const size_t key_unit = (size_t)(b * a.d.key_heads + key_head) * sp.count + pl.at;

    // this wave's rows of K and Q, as planes
    const int row = row_of(w, n16);
    const raw *k_at = (const raw *)a.k + b * a.d.k_batch_stride + key_head * a.d.k_head_stride +
                      (int64_t)(start + (row < here ? row : here - 1)) * a.d.k_step_stride;
    const raw *q_at = (const raw *)a.q + b * a.d.q_batch_stride + key_head * a.d.q_head_stride +
                      (int64_t)(start + (row < here ? row : here - 1)) * a.d.q_step_stride;
    Pack<T, 8> kv[KB], qv[KB];
    auto load = [&](const raw *at, Pack<T, 8> (&v)[KB]) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int col = 32 * kb + 8 * g;
            if (WHOLE) {
                v[kb] = load_pack<T, 8>(at + col);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const raw x = at[col + j < dk ? col + j : dk - 1];
                    v[kb].v[j] = col + j < dk ? x : (raw)0;
                }
            }
        }
    };
    load(k_at, kv);
    load(q_at, qv);
    float beta = 0.0f, log_g = 0.0f;
    if (w == 0 && lane < here) {                // (both under way before either is waited for)
        const int64_t t = start + lane, beta_at = b * a.d.beta_batch_stride + t * a.d.beta_step_stride + head;
        const int64_t g_at = a.g ? b * a.d.g_batch_stride + t * a.d.g_step_stride + head : beta_at;
        auto gates = [&](auto type) {
            using Gate = decltype(type);
            const auto x = ((const typename Gate::raw *)a.beta)[beta_at];
            const auto y = ((const typename Gate::raw *)(a.g ? a.g : a.beta))[g_at];
            beta = Gate::load(x);
            log_g = Gate::load(y);
        };
        if (a.d.gate_dtype == RNN_DTYPE_F32)
            gates(F32{});
        else
            gates(T{});
    }
    v8b kf[KB][KP], qf[KB][KP];
    auto planes = [&](const Pack<T, 8> (&v)[KB], v8b (&out)[KB][KP]) {
        float squares = 0.0f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = row < here ? T::load(v[kb].v[j]) : 0.0f;
            if (a.d.normalize)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    squares = __builtin_fmaf(x[j], x[j], squares);
            const Planes<KP, 8> p(x);
#pragma unroll
            for (int s = 0; s < KP; ++s)
                p.put(s, &out[kb][s]);
        }
        squares += __shfl_xor(squares, 16);
        return squares + __shfl_xor(squares, 32);
    };
    const float kk = planes(kv, kf), qq = planes(qv, qf);
    if (g == 0) {
        rk[row] = key_scale(kk, a.d.normalize);
        rq[row] = key_scale(qq, a.d.normalize) * a.d.scale;
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int p = 0; p < KP; ++p)
            *(v8b *)&keys[p][row][32 * kb + 8 * g] = kf[kb][p];
    if (w == 0) {                               // gates, a step a lane
        double sum = 0.0;
        if (a.g && lane < here)
            sum = log_decay(log_g, a.A != nullptr, a.A ? a.A[head] : 0.0f, a.dt_bias ? a.dt_bias[head] : 0.0f);
        sum = sums_up_to(sum) * 1.4426950408889634074;
        G2[lane] = {(float)sum, (float)(sum - (double)(float)sum)};
        rates[lane] = lane < here ? rate_of(beta, a.d.beta_sigmoid) : 0.0f;
    }
    __syncthreads();
    // (here, where no load is waited for any more: the wait would be for these too)
    if (!DIRECT && head % each == 0) {
        char *to = sp.packed + key_unit * (2 * Sizes::kt) + (size_t)w * KB * KP * kFragment + lane * 16;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                *(v8b *)(to + (kb * KP + p) * kFragment) = kf[kb][p];
                *(v8b *)(to + Sizes::kt + (kb * KP + p) * kFragment) = qf[kb][p];
            }
    }
    auto apart = [&](float2 x, float2 y) { return __builtin_amdgcn_exp2f((x.x - y.x) + (x.y - y.y)); };
    if (w == 3) {
        float *vec = (float *)(sp.vec + unit * Sizes::vec);
        const float2 G = G2[lane];
        const float D = __builtin_amdgcn_exp2f(G.x + G.y);
        vec[place_of(lane)] = D * rk[lane];
        vec[64 + place_of(lane)] = D * rq[lane];
        vec[128 + place_of(lane)] = lane < here ? apart(G2[kChunk - 1], G) * rk[lane] : 0.0f;
        if (lane == kChunk - 1)
            vec[192] = D;
    }

    // L and P, the lower triangle in tiles of 16 columns.  A lane has four of L's rows
    // of a column, and (its operands in the other order) four of P's columns of a row,
    // which are half of what a lane takes of an operand.
    {
        const int i0 = row_of(w, 4 * g);
        float2 Gi[4];
        float fi[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            Gi[r] = G2[i0 + r];
            fi[r] = rates[i0 + r] * rk[i0 + r];
        }
        const float2 Gq = G2[row];
        const float rqi = rq[row];
        char *p_at = sp.p + unit * Sizes::p + (n16 + 16 * (g / 2)) * 16 + g % 2 * 8;
        for (int half = 0; half < (w < 2 ? 1 : 2); ++half) {
            v4f kc[2] = {}, qc[2] = {};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int p = 0; p < KP; ++p)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const v8b other = *(const v8b *)&keys[p][32 * half + 16 * y + n16][32 * kb + 8 * g];
#pragma unroll
                        for (int s = 0; s < KP; ++s)
                            if (s + p <= 2) {
                                kc[y] = mfma(kf[kb][s], other, kc[y]);
                                qc[y] = mfma(other, qf[kb][s], qc[y]);
                            }
                    }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 32 * half + 16 * y + n16, j0 = 32 * half + 16 * y + 4 * g;
                const float2 Gj = G2[j];
                const float rj = rk[j];
                v4f l;
                float p[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    l[r] = j < i0 + r ? fi[r] * (apart(Gi[r], Gj) * rj) * kc[y][r] : 0.0f;
                    p[r] = j0 + r <= row ? rqi * (apart(Gq, G2[j0 + r]) * rk[j0 + r]) * qc[y][r] : 0.0f;
                }
                *(v4f *)&M[j][i0] = l;
                const Planes<PP, 4> out(p);
#pragma unroll
                for (int s = 0; s < PP; ++s)
                    out.put(s, p_at + (size_t)(lower_of(w, half) * PP + s) * kFragment + 32 * y * 16);
            }
        }
    }
    __syncthreads();
    // (1 + L)^-1: the blocks on the diagonal, a column a lane, each entry taken off all
    // below it
    {
        const int at = 16 * w;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            t[i] = i == n16 ? 1.0f : 0.0f;
#pragma unroll
        for (int k = 0; k < 15; ++k) {
            float l[16];
#pragma unroll
            for (int i = (k + 1) / 4 * 4; i < 16; i += 4)
                __builtin_memcpy(&l[i], &M[at + k][at + i], 16);
#pragma unroll
            for (int i = k + 1; i < 16; ++i)
                t[i] = __builtin_fmaf(-l[i], t[k], t[i]);
        }
        // (the wave alone has this block)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            M[at + 4 * g + r][at + n16] = g == 0 ? t[r] : g == 1 ? t[4 + r] : g == 2 ? t[8 + r] : t[12 + r];
    }
    // and those below: T_ij = -T_ii sum_k L_ik T_kj
#pragma unroll
    for (int far = 1; far < 4; ++far) {
        __syncthreads();
        if (w + far < 4) {
            const int i = 16 * (w + far), j = 16 * w;
            v4f x = {}, y = {};
#pragma unroll
            for (int k = 0; k < far; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    x = mfma(M[j + 16 * k + 4 * g + s][i + n16], M[j + 16 * k + 4 * g + s][j + n16], x);
            float own[4];
            __builtin_memcpy(own, &M[i + n16][i + 4 * g], 16);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                y = mfma(own[s], x[s], y);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                M[i + 4 * g + r][j + n16] = -y[r];
        }
    }
    __syncthreads();
    // its operands with the rates, four columns of a row (half of what a lane takes) a time
#pragma unroll
    for (int item = tid; item < 2 * kLower * 64; item += 256) {
        const int f = item / 128, l = item / 2 % 64;
        const int tile = f < 2 ? f : (f + 2) / 2, p = f < 2 ? 0 : f % 2;
        const int i = row_of(tile, l % 16), j = 32 * p + 8 * (l / 16) + 4 * (item % 2);
        float x[4], rate[4];
        __builtin_memcpy(x, &M[i][j], 16);
        __builtin_memcpy(rate, &rates[j], 16);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = j + e <= i ? x[e] * rate[e] : 0.0f;
        const Planes<3, 4> out(x);
        char *to = sp.t + unit * Sizes::t + (size_t)f * 3 * kFragment + l * 16 + item % 2 * 8;
#pragma unroll
        for (int s = 0; s < 3; ++s)
            out.put(s, to + s * kFragment);
    }
    // K transposed: eight steps of a row of the state a lane (by the last of a key head's
    // heads; the first one has left the operands of K and Q)
    if (head % each == each - 1)
        for (int item = tid; item < 4 * KB * 64; item += 256) {
            const int l = item % 64, f = item / 64, tile = f / 2, p = f % 2;
            const int r = row_of(tile, l % 16), i = 32 * p + 8 * (l / 16);
            char *to = sp.kt + key_unit * Sizes::kt + (size_t)f * KP * kFragment + l * 16;
#pragma unroll
            for (int s = 0; s < KP; ++s) {
                v8b x;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = keys[s][i + e][r];
                *(v8b *)(to + s * kFragment) = x;
            }
        }
}

// The waves' accesses to LDS in order; those to global memory stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Orders what stands before it in a phase: reads of LDS, then the products, with the
// loads of coming operands between them.  (A load takes the compute unit about 16
// cycles, and a wave that issues several at once waits for them.)
template <int READS, int PRODUCTS, int LOADS, int I = -1> __device__ __forceinline__ void spread()
{
    constexpr int FIRST = READS < 6 ? READS : 6;
    if constexpr (I < 0) {
        __builtin_amdgcn_sched_group_barrier(0x100, FIRST, 0);
    } else {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if constexpr (I < READS - FIRST)
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        constexpr int LOAD = (I + 1) * LOADS / PRODUCTS - I * LOADS / PRODUCTS;
        if constexpr (LOAD > 0)
            __builtin_amdgcn_sched_group_barrier(0x20, LOAD, 0);
    }
    if constexpr (I + 1 < PRODUCTS)
        spread<READS, PRODUCTS, LOADS, I + 1>();
}
// Products of one operand of KP planes with one of three.
constexpr int kProducts[4] = {0, 3, 5, 6};

// What a wave reads of a chunk.  The first four waves, a tile of its rows each, carry
// the state along; four others, beside them, make the outputs.
// Tiles 0 and 1 have one operand of a lower triangle (N = 1), 2 and 3 two.
template <class T, int KB, int N> struct StateOperands {
    static constexpr int KP = kPlanes<T>, TW = (2 * KB + 3) / 4;
    v8b k[KB][KP], t[N][3], kt[TW][2][KP];
    static constexpr int registers = 4 * (KB * KP + 6 + 2 * TW * KP);
};
template <class T, int KB, int N, int NC> struct OutOperands {
    static constexpr int KP = kPlanes<T>, PP = kOutLast<T> + 1;
    v8b q[KB][KP], p[N][PP];
    typedef uint32_t Four __attribute__((ext_vector_type(sizeof(typename T::raw))));    // values
    v4f vec;
    Four v[NC];
    static constexpr int registers = 4 * (KB * KP + 2 * PP) + 4 + NC * (int)sizeof(typename T::raw);
};
// Two chunks are on their way where the registers of a wave (256) hold them.
template <class Operands> constexpr int kAhead = Operands::registers <= 90 ? 2 : 1;

// f(operands of the chunk, of the one before it, chunk, the chunk whose operands take
// its own's place, whether all its steps are there for sure) for each chunk of [first,
// last).
template <int AHEAD, bool WHOLE, class Operands, class Load, class F>
__device__ __forceinline__ void along(int first, int last, Operands (&x)[AHEAD], Load &&load, F &&f)
{
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        load(x[i], first + i < last ? first + i : last - 1);
    lds_barrier();                              // (the state is published)
    int c = first;
    for (; c + AHEAD < last; c += AHEAD)        // (no way round a load: waits are by their number)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            f(x[i], x[(i + AHEAD - 1) % AHEAD], c + i, c + i + AHEAD < last ? c + i + AHEAD : last - 1,
              std::integral_constant<bool, WHOLE>{});
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (c + i < last)
            f(x[i], x[(i + AHEAD - 1) % AHEAD], c + i, last - 1, std::false_type{});
}

// NC tiles of 16 columns of the state a workgroup.
template <class T, int KB, bool DIRECT, int NC>
__global__ __launch_bounds__(512) void delta_chunks_kernel(DeltaArgs a, DeltaSpan sp, uint32_t slices)
{
    using raw = typename T::raw;
    using Sizes = DeltaSizes<T, KB>;
    constexpr int KP = kPlanes<T>, LAST = kOutLast<T>, PP = LAST + 1, TILES = 2 * KB, TW = (TILES + 3) / 4;
    __shared__ v8b Sf[NC][KB][3][64], Rf[NC][2][3][64], Uf[NC][2][PP][64], Wf[NC][2][3][64];
    __shared__ v4f rows[2][64];                 // factors of rows of this chunk and the next
    __shared__ __attribute__((aligned(16))) raw Vs[kChunk][16 * NC];
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), w = wave % 4;
    const int n16 = lane % 16, g = lane / 16;
    const Place pl = place_in(slices);
    const uint32_t heads = (uint32_t)a.d.heads;
    const int64_t b = pl.bh / heads, head = pl.bh % heads;
    if (b >= a.d.batch)
        return;
    const int n = delta_steps(a, b), steps = (int)a.d.steps;
    const int dk = (int)a.d.key_dim, dv = (int)a.d.value_dim, col0 = (int)pl.at * 16 * NC, col = col0 + n16;
    const bool all_in = col0 + 16 * NC <= dv;
    const int64_t key_head = head / (a.d.heads / a.d.key_heads);
    const int first = (int)sp.first, all = (n + kChunk - 1) / kChunk;
    const int last = first + (int)sp.count < all ? first + (int)sp.count : all;     // chunks [first, last)

    // Addresses: a base for all lanes that moves along, and 32 bits of a lane (the rows of
    // 64 steps span less than 2^31 bytes).
    const int row = row_of(w, n16), out_row = row_of(w, 4 * g);
    char *o_at = (char *)a.o + (b * a.d.o_batch_stride + head * a.d.o_head_stride) * sizeof(raw);
    const uint32_t o_step = (uint32_t)a.d.o_step_stride * sizeof(raw);
    const uint32_t o_col = (uint32_t)col * sizeof(raw);
    const size_t unit0 = (size_t)pl.bh * sp.count;
    const size_t key_unit0 = (size_t)(b * a.d.key_heads + key_head) * sp.count;
    const uint32_t lane16 = lane * 16;
    const int row4 = 4 * w + g;                 // of `rows`: this lane's four rows
    auto operand = [&](const char *base) { return *(const v8b *)(base + lane16); };
    auto vec_of = [&](int c) { return sp.vec + (unit0 + c - first) * Sizes::vec; };
    // This wave's rows of K (0) or Q (1).
    auto load_rows = [&](const void *base, int64_t bs, int64_t ss, int64_t hs, int which, int c, v8b (&x)[KB][KP]) {
        if (DIRECT) {
            const int most = n - 1 - kChunk * c;        // the last row of the chunk that is there
            const uint32_t step = (uint32_t)ss * sizeof(raw), at = (row < most ? row : most) * step + 16 * g;
            const char *from = (const char *)base + (b * bs + key_head * hs) * sizeof(raw) + (size_t)c * kChunk * step;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                x[kb][0] = __builtin_bit_cast(v8b, load_pack<BF16, 8>((const uint16_t *)(from + at) + 32 * kb));
        } else {
            const char *at = sp.packed + (key_unit0 + c - first) * (2 * Sizes::kt) + which * Sizes::kt +
                             (size_t)w * KB * KP * kFragment;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int p = 0; p < KP; ++p)
                    x[kb][p] = operand(at + (kb * KP + p) * kFragment);
        }
    };
    // Operands of a lower triangle.
    auto load_lower = [&](const char *at, auto &x) {
        constexpr int N = sizeof(x) / sizeof(x[0]), P = sizeof(x[0]) / sizeof(v8b);
#pragma unroll
        for (int p = 0; p < N; ++p)
#pragma unroll
            for (int s = 0; s < P; ++s)
                x[p][s] = operand(at + (size_t)(lower_of(w, p) * P + s) * kFragment);
    };

    // (Tiles with one and with two operands of a triangle go their own ways: a branch
    // around some of a wave's products loses the wait that reading the others' results
    // needs.)
    auto carry = [&](auto operands) {
        // the state: this wave's tiles in registers, everyone's as operands in LDS
        constexpr int N = decltype(operands)::value;
        using Operands = StateOperands<T, KB, N>;
        v4f S[NC][TW];
        const int64_t state_at = (int64_t)pl.bh * dk * dv + col;
#pragma unroll
        for (int z = 0; z < NC; ++z)
#pragma unroll
            for (int x = 0; x < TW; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = row_of(w * TW + x, 4 * g + r);
                    S[z][x][r] = sp.from && col + 16 * z < dv && at < dk
                                     ? sp.from[state_at + (int64_t)at * dv + 16 * z] : 0.0f;
                }
        auto publish = [&]() {
#pragma unroll
            for (int z = 0; z < NC; ++z)
#pragma unroll
                for (int x = 0; x < TW; ++x) {
                    const int tile = w * TW + x;
                    const float s[4] = {S[z][x][0], S[z][x][1], S[z][x][2], S[z][x][3]};
                    const Planes<3, 4> out(s);
                    if (4 * TW == TILES || tile < TILES)
#pragma unroll
                        for (int p = 0; p < 3; ++p)
                            out.put(p, (v4b *)&Sf[z][tile / 2][p][lane] + tile % 2);
                }
        };
        auto load_k = [&](Operands &x, int c) {
            load_rows(a.k, a.d.k_batch_stride, a.d.k_step_stride, a.d.k_head_stride, 0, c, x.k);
        };
        auto load_t = [&](Operands &x, int c) { load_lower(sp.t + (unit0 + c - first) * Sizes::t, x.t); };
        auto load_kt = [&](Operands &x, int c) {
            const char *at = sp.kt + (key_unit0 + c - first) * Sizes::kt;
#pragma unroll
            for (int y = 0; y < TW; ++y) {
                const int tile = w * TW + y < TILES ? w * TW + y : TILES - 1;
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int s = 0; s < KP; ++s)
                        x.kt[y][p][s] = operand(at + (size_t)((tile * 2 + p) * KP + s) * kFragment);
            }
        };
        __builtin_amdgcn_s_setprio(3);
        if (first < last) {
            publish();
            constexpr int AHEAD = kAhead<Operands>;
            Operands both[AHEAD];
            along<AHEAD, true>(first, last, both, [&](Operands &x, int c) {
                load_k(x, c);
                load_t(x, c);
                load_kt(x, c);
            }, [&](Operands &x, Operands &before, int c, int next, auto) {
                // K S, and what the corrections solve for
                load_kt(before, c + AHEAD - 1 < last ? c + AHEAD - 1 : last - 1);
                v4f X[NC][2] = {};
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int p = 0; p < 3; ++p)
#pragma unroll
                        for (int z = 0; z < NC; ++z) {
                            const v8b s = Sf[z][kb][p][lane];
#pragma unroll
                            for (int e = 0; e + p <= 2 && e < KP; ++e)
                                X[z][e + p > 0] = mfma(x.k[kb][e], s, X[z][e + p > 0]);
                        }
                spread<3 * KB * NC, KB * kProducts[KP] * NC, 2 * TW * KP>();
                const v4f k_row = rows[c % 2][row4];
#pragma unroll
                for (int z = 0; z < NC; ++z) {
                    float R[4];                 // (T has zeros for rows that are not there)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        R[r] = __builtin_fmaf(-k_row[r], X[z][1][r] + X[z][0][r],
                                              T::load(Vs[out_row + r][16 * z + n16]));
                    const Planes<3, 4> r_out(R);
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        r_out.put(p, (v4b *)&Rf[z][w / 2][p][lane] + w % 2);
                }
                lds_barrier();
                // the corrections
                v4f u[NC][2] = {};
#pragma unroll
                for (int p = 0; p < N; ++p)
#pragma unroll
                    for (int s = 0; s < 3; ++s)
#pragma unroll
                        for (int z = 0; z < NC; ++z) {
                            const v8b r = Rf[z][p][s][lane];
#pragma unroll
                            for (int e = 0; e + s <= 2; ++e)
                                u[z][e + s > 0] = mfma(x.t[p][e], r, u[z][e + s > 0]);
                        }
                load_k(x, next);
                spread<3 * N * NC, 6 * N * NC, KB * KP>();
                const v4f w_row = rows[c % 2][32 + row4];
#pragma unroll
                for (int z = 0; z < NC; ++z) {
                    float U[4], W[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        U[r] = u[z][1][r] + u[z][0][r];
                        W[r] = U[r] * w_row[r];
                    }
                    const Planes<3, 4> w_out(W);
                    const Planes<PP, 4> u_out(U);
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        w_out.put(p, (v4b *)&Wf[z][w / 2][p][lane] + w % 2);
#pragma unroll
                    for (int p = 0; p < PP; ++p)
                        u_out.put(p, (v4b *)&Uf[z][w / 2][p][lane] + w % 2);
                }
                lds_barrier();
                // the state
                v4f d[NC][TW][2] = {};
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int s = 0; s < 3; ++s)
#pragma unroll
                        for (int z = 0; z < NC; ++z) {
                            const v8b f = Wf[z][p][s][lane];
#pragma unroll
                            for (int t = 0; t < TW; ++t)
#pragma unroll
                                for (int e = 0; e + s <= 2 && e < KP; ++e)
                                    d[z][t][e + s > 0] = mfma(x.kt[t][p][e], f, d[z][t][e + s > 0]);
                        }
                load_t(x, next);
                spread<6 * NC, 2 * TW * kProducts[KP] * NC, 3 * N>();
                const float D = rows[c % 2][48][0];
#pragma unroll
                for (int z = 0; z < NC; ++z)
#pragma unroll
                    for (int t = 0; t < TW; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            S[z][t][r] = __builtin_fmaf(D, S[z][t][r], d[z][t][1][r] + d[z][t][0][r]);
                publish();
                lds_barrier();
            });
        }
#pragma unroll
        for (int z = 0; z < NC; ++z)
#pragma unroll
            for (int x = 0; x < TW; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = row_of(w * TW + x, 4 * g + r);
                    if (sp.to && col + 16 * z < dv && at < dk)
                        sp.to[state_at + (int64_t)at * dv + 16 * z] = S[z][x][r];
                }
    };

    // the outputs; values and factors of rows are brought into LDS.  WHOLE: all columns
    // are there.  (Where the number of loads and stores under way depends on a branch, all
    // of them are waited for: whole chunks have no such branch.)
    auto answer = [&](auto operands, auto whole) {
        constexpr int N = decltype(operands)::value;
        constexpr bool WHOLE = decltype(whole)::value;
        using Operands = OutOperands<T, KB, N, NC>;
        constexpr int AHEAD = kAhead<Operands>;
        const char *v_at = (const char *)a.v + (b * a.d.v_batch_stride + head * a.d.v_head_stride) * sizeof(raw);
        const uint32_t v_step = (uint32_t)a.d.v_step_stride * sizeof(raw);
        const int v_row = 16 * w + lane / 4, v_col = col0 + 4 * (lane % 4);
        auto load_q = [&](Operands &x, int c) {
            load_rows(a.q, a.d.q_batch_stride, a.d.q_step_stride, a.d.q_head_stride, 1, c, x.q);
        };
        auto load_p = [&](Operands &x, int c) { load_lower(sp.p + (unit0 + c - first) * Sizes::p, x.p); };
        // Of the chunk after c.  (All factors by every one of the four waves, so that none
        // goes its own way.)
        auto load_vec = [&](Operands &x, int c) {
            x.vec = *(const v4f *)(vec_of(c + 1 < last ? c + 1 : last - 1) + lane16);
        };
        auto load_v = [&](Operands &x, int c) {
            c = c + 1 < last ? c + 1 : last - 1;
            const int most = n - 1 - kChunk * c;
            const char *at = v_at + (size_t)c * kChunk * v_step;
            const uint32_t row = (uint32_t)(v_row < most ? v_row : most) * v_step;
#pragma unroll
            for (int z = 0; z < NC; ++z) {
                const int at_col = v_col + 16 * z;
                typename Operands::Four v = {};
                if (WHOLE) {
                    __builtin_memcpy(&v, at + (row + at_col * (uint32_t)sizeof(raw)), sizeof(v));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int there = at_col + j < dv ? at_col + j : dv - 1;
                        const uint32_t r = *(const raw *)(at + (row + there * (uint32_t)sizeof(raw)));
                        v[j * sizeof(raw) / 4] |= sizeof(raw) == 4 ? r : r << 16 * (j % 2);
                    }
                }
                x.v[z] = v;
            }
        };
        auto put_v = [&](const Operands &x) {
#pragma unroll
            for (int z = 0; z < NC; ++z)
                *(typename Operands::Four *)&Vs[v_row][16 * z + 4 * (lane % 4)] = x.v[z];
        };
        // (Operands are replaced where these waves have nothing else to do: a load waits for
        // those before it, and a barrier for the wave.)
        auto chunk = [&](Operands &x, Operands &before, int c, int next, auto all_rows) {
            rows[(c + 1) % 2][lane] = x.vec;
            load_vec(x, next);
            load_p(before, c + AHEAD - 1 < last ? c + AHEAD - 1 : last - 1);
            const v4f q_row = rows[c % 2][16 + row4];
            lds_barrier();
            v4f Y[NC][2] = {}, O[NC][2] = {};   // Q S, while the corrections are made
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int p = 0; p <= LAST; ++p)
#pragma unroll
                    for (int z = 0; z < NC; ++z) {
                        const v8b s = Sf[z][kb][p][lane];
#pragma unroll
                        for (int e = 0; e + p <= LAST && e < KP; ++e)
                            Y[z][e + p > 0] = mfma(x.q[kb][e], s, Y[z][e + p > 0]);
                    }
            put_v(x);
            load_v(x, next);
            load_q(x, next);
            lds_barrier();
#pragma unroll
            for (int y = 0; y < N; ++y)
#pragma unroll
                for (int s = 0; s < PP; ++s)
#pragma unroll
                    for (int z = 0; z < NC; ++z) {
                        const v8b f = Uf[z][y][s][lane];
#pragma unroll
                        for (int e = 0; e + s <= LAST; ++e)
                            O[z][e + s > 0] = mfma(x.p[y][e], f, O[z][e + s > 0]);
                    }
            char *to = o_at + (size_t)c * kChunk * o_step;
            const int start = kChunk * c;
#pragma unroll
            for (int z = 0; z < NC; ++z)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const raw out = T::store(__builtin_fmaf(q_row[r], Y[z][1][r] + Y[z][0][r], O[z][1][r] + O[z][0][r]));
                    if (decltype(all_rows)::value || (col + 16 * z < dv && start + out_row + r < n))
                        *(raw *)(to + ((out_row + r) * o_step + o_col + 16 * z * (uint32_t)sizeof(raw))) = out;
                }
            lds_barrier();
        };
        if (first < last) {
            Operands x[AHEAD];
            load_vec(x[0], first - 1);
            load_v(x[0], first - 1);
            rows[first % 2][lane] = x[0].vec;
            put_v(x[0]);
            along<AHEAD, WHOLE>(first, last, x, [&](Operands &y, int c) {
                load_vec(y, c);
                load_v(y, c);
                load_q(y, c);
                load_p(y, c);
            }, chunk);
        }
    };
    if (wave < 4) {
        if (w < 2)
            carry(std::integral_constant<int, 1>{});
        else
            carry(std::integral_constant<int, 2>{});
        return;
    }
    if (all_in) {
        if (w < 2)
            answer(std::integral_constant<int, 1>{}, std::true_type{});
        else
            answer(std::integral_constant<int, 2>{}, std::true_type{});
    } else {
        if (w < 2)
            answer(std::integral_constant<int, 1>{}, std::false_type{});
        else
            answer(std::integral_constant<int, 2>{}, std::false_type{});
    }
    // steps behind the last one of this span: zeros
    const int from = n > kChunk * first ? n : kChunk * first;
    const int64_t to = (int64_t)kChunk * (first + (int64_t)sp.count);
    const int until = to < steps ? (int)to : steps;
#pragma unroll
    for (int z = 0; z < NC; ++z)
        if (col + 16 * z < dv)
            for (int t = from + (tid - 256) / 16; t < until; t += 16)
                *(raw *)(o_at + (size_t)t * o_step + o_col + 16 * z * sizeof(raw)) = 0;
}

// The workspace of a span of `count` chunks, as its parts lie in it; then the
// states between spans where the caller wants none at the end.
struct DeltaLayout {
    size_t t, p, vec, kt, packed, states, all;
};
template <class T, int KB> static DeltaLayout layout_of(const rnn_delta_desc &d, uint64_t count, bool direct)
{
    using Sizes = DeltaSizes<T, KB>;
    const size_t units = (size_t)d.batch * d.heads * count, key_units = (size_t)d.batch * d.key_heads * count;
    DeltaLayout l;
    l.t = 0;
    l.p = l.t + units * Sizes::t;
    l.vec = l.p + units * Sizes::p;
    l.kt = l.vec + units * Sizes::vec;
    l.packed = l.kt + key_units * Sizes::kt;
    l.states = l.packed + (direct ? 0 : key_units * 2 * Sizes::kt);
    l.all = l.states;
    return l;
}
static uint64_t chunks_of(const rnn_delta_desc &d) { return ((uint64_t)d.steps + kChunk - 1) / kChunk; }

// Chunks that are prepared at once: all, or as many as 256 MB of workspace hold (the
// last-level cache, where the second kernel finds them).  8 rows of 1024 steps of 32 heads
// (128 x 128, bf16): 280 us so and with 1 GB, 349 us with 64 MB, whose last waves of
// workgroups are a larger part; in f32 one row of 4096 steps 370 us (3 launches of each
// kernel), with 1 GB 372.
constexpr size_t kMostWorkspace = (size_t)256 << 20;
template <class T, int KB> static uint64_t span_of(const rnn_delta_desc &d, bool direct)
{
    const uint64_t all = chunks_of(d), most = kMostWorkspace / layout_of<T, KB>(d, 1, direct).all;
    return most < 1 ? 1 : most < all ? most : all;
}

// Two tiles of columns a workgroup where one would be more workgroups than compute
// units: a workgroup's chain is longer, but the operands are read half as often.  The
// second kernel, bf16, 128 x 128, two against one: 2 rows of 4096 steps of 32 heads 180 us
// against 255, 8 of 1024 201 and 284, one of 48 heads 342 and 460; one of 32 heads (256
// workgroups) 320 and 245.  f32, 64 x 64, 8 rows of 1000 steps: 16 heads 70 and 100, 8
// heads (256) 38 and 31.  Keys beyond 192 do not fit the registers twice.
static bool wide_slices(const rnn_delta_desc &d)
{
    return d.key_dim <= 192 && d.batch * d.heads * ((d.value_dim + 15) / 16) > 256;
}

template <class T, int KB, bool DIRECT> static int chunks_go(const DeltaArgs &a, hipStream_t s)
{
    const uint64_t all = chunks_of(a.d), span = span_of<T, KB>(a.d, DIRECT);
    const DeltaLayout l = layout_of<T, KB>(a.d, span, DIRECT);
    const uint64_t rounds = ((uint64_t)a.d.batch * a.d.heads + 7) / 8;
    const bool wide = wide_slices(a.d);
    const uint64_t slices = ((uint64_t)a.d.value_dim + (wide ? 31 : 15)) / (wide ? 32 : 16);
    if (!launchable(rounds * 8 * span, 256) || !launchable(rounds * 8 * slices, 512))
        return (int)hipErrorInvalidConfiguration;
    char *ws = (char *)a.workspace;
    float *between = a.state_out ? a.state_out : span < all ? (float *)(ws + l.states) : nullptr;
    for (uint64_t first = 0; first < all; first += span) {
        const uint64_t count = all - first < span ? all - first : span;
        const DeltaSpan sp{(uint32_t)first, (uint32_t)count, ws + l.t, ws + l.p, ws + l.vec, ws + l.kt,
                           ws + l.packed, first == 0 ? a.state_in : between, between};
        const dim3 units((uint32_t)(rounds * 8 * count));
        if (DIRECT || a.d.key_dim == 32 * KB)
            delta_prepare_kernel<T, KB, DIRECT, true><<<units, dim3(256), 0, s>>>(a, sp);
        else if constexpr (!DIRECT)
            delta_prepare_kernel<T, KB, DIRECT, false><<<units, dim3(256), 0, s>>>(a, sp);
        int rc = (int)hipGetLastError();
        if (rc)
            return rc;
        const dim3 grid((uint32_t)(rounds * 8 * slices)), block(512);
        if constexpr (!DIRECT)
            if (!wide)
                delta_chunks_kernel<T, KB, DIRECT, 1><<<grid, block, 0, s>>>(a, sp, (uint32_t)slices);
        if constexpr (KB <= 6)
            if (wide)
                delta_chunks_kernel<T, KB, DIRECT, 2><<<grid, block, 0, s>>>(a, sp, (uint32_t)slices);
        rc = (int)hipGetLastError();
        if (rc)
            return rc;
    }
    return 0;
}

// f(type, blocks of 32 rows of the state, whether keys and queries are read as they are:
// bfloat16 of whole blocks, where two tiles of columns share what is read).  Elsewhere the
// first kernel leaves them as operands, one after another: it writes more, but a head's
// rows lie kilobytes apart, and each of its workgroups reads them all.  Both kernels, as
// operands against as they are, bf16: one row of 32 heads over 16, 8192 steps 326 us
// against 347, over 8, 4096 steps 129 and 155; 4 heads of 256 x 256, 4096 steps 170 and 213;
// two tiles at a time 8 rows of 1024 steps 277 and 274, 2 of 4096 steps and 32 key heads
// 297 and 275.
template <class F> static auto with_sizes(const rnn_delta_desc &d, F &&f)
{
    auto blocks = [&](auto type) {
        using T = decltype(type);
        auto at = [&](auto kb) {
            constexpr int KB = decltype(kb)::value;
            if constexpr (std::is_same<T, BF16>::value && KB <= 6)
                if (d.key_dim == 32 * KB && wide_slices(d))
                    return f(type, kb, std::true_type{});
            return f(type, kb, std::false_type{});
        };
        const int64_t kb = (d.key_dim + 31) / 32;
        if (kb <= 1)
            return at(std::integral_constant<int, 1>{});
        if (kb == 2)
            return at(std::integral_constant<int, 2>{});
        if (kb == 3)
            return at(std::integral_constant<int, 3>{});
        if (kb == 4)
            return at(std::integral_constant<int, 4>{});
        return kb <= 6 ? at(std::integral_constant<int, 6>{}) : at(std::integral_constant<int, 8>{});
    };
    switch (d.dtype) {
    case RNN_DTYPE_F32: return blocks(F32{});
    case RNN_DTYPE_BF16: return blocks(BF16{});
    default: return blocks(F16{});
    }
}

size_t delta_chunks_workspace(const rnn_delta_desc &d)
{
    return with_sizes(d, [&](auto type, auto kb, auto direct) -> size_t {
        using T = decltype(type);
        constexpr int KB = decltype(kb)::value;
        const uint64_t span = span_of<T, KB>(d, direct.value);
        const size_t between = span < chunks_of(d)
                                   ? (size_t)d.batch * d.heads * d.key_dim * d.value_dim * sizeof(float)
                                   : 0;
        return layout_of<T, KB>(d, span, direct.value).all + between;
    });
}

int launch_delta_chunks(const DeltaArgs &a, hipStream_t s)
{
    return with_sizes(a.d, [&](auto type, auto kb, auto direct) -> int {
        return chunks_go<decltype(type), decltype(kb)::value, decltype(direct)::value>(a, s);
    });
}

}  // namespace rnnamd
