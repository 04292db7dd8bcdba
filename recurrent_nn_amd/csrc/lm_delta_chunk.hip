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

// Plane p of x, taken off it.
__device__ __forceinline__ __bf16 next_plane(float &x)
{
    const __bf16 p = (__bf16)x;
    x -= (float)p;
    return p;
}
template <int P> __device__ __forceinline__ void planes_of(const float (&x)[8], v8b (&out)[P])
{
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        rest[j] = x[j];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            out[p][j] = next_plane(rest[j]);
}

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
constexpr int kVec = 512;               // floats: e^G |k|, scale e^G |q|, e^(G_63 - G) |k|, e^G_63; zeros
constexpr int kZeros = 256;             // an operand of zeros

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

template <class T, int KB, bool DIRECT>
__global__ __launch_bounds__(256) void delta_prepare_kernel(DeltaArgs a, DeltaSpan sp)
{
    using raw = typename T::raw;
    constexpr int KP = kPlanes<T>, PP = kOutLast<T> + 1, LDK = 32 * KB + 8, LDT = 68;
    using Sizes = DeltaSizes<T, KB>;
    __shared__ __attribute__((aligned(16))) __bf16 keys[KP][kChunk][LDK];
    __shared__ __attribute__((aligned(16))) float Lm[kChunk][LDT], Pm[kChunk][LDT], Tm[kChunk][LDT];
    __shared__ float2 G2[kChunk];
    __shared__ float rates[kChunk], rk[kChunk], rq[kChunk];
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
    auto load = [&](const void *base, int64_t bs, int64_t ss, int64_t hs, v8b (&out)[KB][KP]) {
        const raw *at = (const raw *)base + b * bs + key_head * hs +
                        (int64_t)(start + (row < here ? row : here - 1)) * ss;
        float squares = 0.0f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int col = 32 * kb + 8 * g;
            float x[8];
            if (DIRECT || dk == 32 * KB) {
                const Pack<T, 8> v = load_pack<T, 8>(at + col);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = T::load(v.v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = T::load(at[col + j < dk ? col + j : dk - 1]);
                    x[j] = col + j < dk ? v : 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = row < here ? x[j] : 0.0f;
                squares = __builtin_fmaf(x[j], x[j], squares);
            }
            planes_of<KP>(x, out[kb]);
        }
        squares += __shfl_xor(squares, 16);
        return squares + __shfl_xor(squares, 32);
    };
    v8b kf[KB][KP], qf[KB][KP];
    const float kk = load(a.k, a.d.k_batch_stride, a.d.k_step_stride, a.d.k_head_stride, kf);
    const float qq = load(a.q, a.d.q_batch_stride, a.d.q_step_stride, a.d.q_head_stride, qf);
    if (g == 0) {
        rk[row] = key_scale(kk, a.d.normalize);
        rq[row] = key_scale(qq, a.d.normalize) * a.d.scale;
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int p = 0; p < KP; ++p)
            *(v8b *)&keys[p][row][32 * kb + 8 * g] = kf[kb][p];
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
    if (w == 0) {                               // gates, a step a lane
        float decay = 0.0f, rate = 0.0f;
        if (lane < here) {
            const int64_t t = start + lane;
            rate = rate_of(gate_at<T>(a.beta, a.d.gate_dtype,
                                      b * a.d.beta_batch_stride + t * a.d.beta_step_stride + head),
                           a.d.beta_sigmoid);
            if (a.g)
                decay = log_decay(gate_at<T>(a.g, a.d.gate_dtype,
                                             b * a.d.g_batch_stride + t * a.d.g_step_stride + head),
                                  a.A != nullptr, a.A ? a.A[head] : 0.0f, a.dt_bias ? a.dt_bias[head] : 0.0f);
        }
        double sum = decay;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double before = __shfl_up(sum, d);
            sum += lane >= d ? before : 0.0;
        }
        G2[lane] = {(float)sum, (float)(sum - (double)(float)sum)};
        rates[lane] = rate;
    }
    __syncthreads();
    auto apart = [&](float2 x, float2 y) { return expf((x.x - y.x) + (x.y - y.y)); };
    if (tid < kChunk) {
        float *vec = (float *)(sp.vec + unit * Sizes::vec);
        const float2 G = G2[tid];
        const float D = expf(G.x + G.y);
        vec[place_of(tid)] = D * rk[tid];
        vec[64 + place_of(tid)] = D * rq[tid];
        vec[128 + place_of(tid)] = tid < here ? apart(G2[kChunk - 1], G) * rk[tid] : 0.0f;
        if (tid == kChunk - 1)
            vec[192] = D;
        *(v4f *)(vec + kZeros + 4 * tid) = v4f{};
    }

    // L and P, the lower triangle in tiles of 16 columns
    for (int c = 0; c < (w < 2 ? 2 : 4); ++c) {
        v4f kc = {}, qc = {};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                const v8b other = *(const v8b *)&keys[p][16 * c + n16][32 * kb + 8 * g];
#pragma unroll
                for (int s = 0; s < KP; ++s)
                    if (s + p <= 2) {
                        kc = mfma(kf[kb][s], other, kc);
                        qc = mfma(qf[kb][s], other, qc);
                    }
            }
        const int j = 16 * c + n16;
        const float2 Gj = G2[j];
        const float rj = rk[j];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = row_of(w, 4 * g + r);
            const float e = apart(G2[i], Gj) * rj;
            Lm[i][j] = j < i ? rates[i] * rk[i] * e * kc[r] : 0.0f;
            Pm[i][j] = j <= i ? rq[i] * e * qc[r] : 0.0f;
        }
    }
    __syncthreads();
    // (1 + L)^-1: the blocks on the diagonal, a column a lane
    {
        const int at = 16 * w;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            t[i] = i == n16 ? 1.0f : 0.0f;
#pragma unroll
            for (int k = 0; k < i; ++k)
                t[i] = __builtin_fmaf(-Lm[at + i][at + k], t[k], t[i]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i / 4 == g)
                Tm[at + i][at + n16] = t[i];
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
                    x = mfma(Lm[i + n16][j + 16 * k + 4 * g + s], Tm[j + 16 * k + 4 * g + s][j + n16], x);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                y = mfma(Tm[i + n16][i + 4 * g + s], x[s], y);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                Tm[i + 4 * g + r][j + n16] = -y[r];
        }
    }
    __syncthreads();
    // operands of the lower triangles, eight columns of a row a lane
    for (int item = tid; item < kLower * 64; item += 256) {
        const int f = item / 64, l = item % 64;
        const int tile = f < 2 ? f : (f + 2) / 2, p = f < 2 ? 0 : f % 2;
        const int i = row_of(tile, l % 16), j = 32 * p + 8 * (l / 16);
        float x[8];
        v8b tp[3], pp[PP];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = j + e <= i ? Tm[i][j + e] * rates[j + e] : 0.0f;
        planes_of<3>(x, tp);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = Pm[i][j + e];
        planes_of<PP>(x, pp);
        char *to = sp.t + unit * Sizes::t + (size_t)f * 3 * kFragment + l * 16;
#pragma unroll
        for (int s = 0; s < 3; ++s)
            *(v8b *)(to + s * kFragment) = tp[s];
        to = sp.p + unit * Sizes::p + (size_t)f * PP * kFragment + l * 16;
#pragma unroll
        for (int s = 0; s < PP; ++s)
            *(v8b *)(to + s * kFragment) = pp[s];
    }
    // K transposed: eight steps of a row of the state a lane
    if (head % each == 0)
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

template <class T, int KB, bool DIRECT>
__global__ __launch_bounds__(256) void delta_chunks_kernel(DeltaArgs a, DeltaSpan sp, uint32_t slices)
{
    using raw = typename T::raw;
    using Sizes = DeltaSizes<T, KB>;
    constexpr int KP = kPlanes<T>, LAST = kOutLast<T>, PP = LAST + 1, TILES = 2 * KB, TW = (TILES + 3) / 4;
    __shared__ v8b Sf[KB][3][64], Rf[2][3][64], Uf[2][PP][64], Wf[2][3][64];
    const int tid = threadIdx.x, lane = tid % 64, w = __builtin_amdgcn_readfirstlane(tid / 64);
    const int n16 = lane % 16, g = lane / 16;
    const Place pl = place_in(slices);
    const uint32_t heads = (uint32_t)a.d.heads;
    const int64_t b = pl.bh / heads, head = pl.bh % heads;
    if (b >= a.d.batch)
        return;
    const int n = delta_steps(a, b), steps = (int)a.d.steps;
    const int dk = (int)a.d.key_dim, dv = (int)a.d.value_dim, col = (int)pl.at * 16 + n16;
    const bool in = col < dv;
    const int64_t key_head = head / (a.d.heads / a.d.key_heads);
    const int first = (int)sp.first, all = (n + kChunk - 1) / kChunk;
    const int last = first + (int)sp.count < all ? first + (int)sp.count : all;     // chunks [first, last)

    // the state: this wave's tiles in registers, everyone's as operands in LDS
    v4f S[TW];
    const int64_t state_at = (int64_t)pl.bh * dk * dv + col;
    auto publish = [&]() {
#pragma unroll
        for (int x = 0; x < TW; ++x) {
            const int tile = w * TW + x;
            if (tile < TILES) {
                v4f rest = S[x];
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    v4b out;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        out[r] = next_plane(((float *)&rest)[r]);
                    ((v4b *)&Sf[tile / 2][p][lane])[tile % 2] = out;
                }
            }
        }
    };
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = row_of(w * TW + x, 4 * g + r);
            S[x][r] = sp.from && in && row < dk ? sp.from[state_at + (int64_t)row * dv] : 0.0f;
        }

    const int row = row_of(w, n16), out_row = row_of(w, 4 * g);
    const raw *k_at = (const raw *)a.k + b * a.d.k_batch_stride + key_head * a.d.k_head_stride;
    const raw *q_at = (const raw *)a.q + b * a.d.q_batch_stride + key_head * a.d.q_head_stride;
    const raw *v_at = (const raw *)a.v + b * a.d.v_batch_stride + head * a.d.v_head_stride + (in ? col : dv - 1);
    raw *o_at = (raw *)a.o + b * a.d.o_batch_stride + head * a.d.o_head_stride + col;
    const size_t unit0 = (size_t)pl.bh * sp.count;
    const size_t key_unit0 = (size_t)(b * a.d.key_heads + key_head) * sp.count;

    v8b kf[KB][KP], qf[KB][KP], tf[2][3], pf[2][PP], ktf[TW][2][KP];
    raw v[4];
    v4f dk_row, dq_row, w_row;
    float D;
    auto load_rows = [&](int c) {
        if (DIRECT) {
            const int t = kChunk * c + row;
            const int64_t at = t < n ? t : n - 1;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                kf[kb][0] = __builtin_bit_cast(v8b, load_pack<T, 16 / sizeof(raw)>(
                                                        k_at + at * a.d.k_step_stride + 32 * kb + 8 * g));
                qf[kb][0] = __builtin_bit_cast(v8b, load_pack<T, 16 / sizeof(raw)>(
                                                        q_at + at * a.d.q_step_stride + 32 * kb + 8 * g));
            }
        } else {
            const char *at = sp.packed + (key_unit0 + c - first) * (2 * Sizes::kt) +
                             (size_t)w * KB * KP * kFragment + lane * 16;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    kf[kb][p] = *(const v8b *)(at + (kb * KP + p) * kFragment);
                    qf[kb][p] = *(const v8b *)(at + Sizes::kt + (kb * KP + p) * kFragment);
                }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = kChunk * c + out_row + r;
            v[r] = v_at[(int64_t)(t < n ? t : n - 1) * a.d.v_step_stride];
        }
    };
    auto load_vec = [&](int c) {
        const float *vec = (const float *)(sp.vec + (unit0 + c - first) * Sizes::vec);
        dk_row = *(const v4f *)(vec + 16 * w + 4 * g);
        dq_row = *(const v4f *)(vec + 64 + 16 * w + 4 * g);
        w_row = *(const v4f *)(vec + 128 + 16 * w + 4 * g);
        D = vec[192];
    };
    // Tiles 0 and 1 have nothing beyond the diagonal: zeros in the place of a second
    // operand, since a branch around its products loses the wait that reading the
    // others' results needs.
    auto lower = [&](const char *at, const char *zeros, int p, int s, int planes) {
        return *(const v8b *)(p == 1 && w < 2 ? zeros : at + (size_t)(lower_of(w, p) * planes + s) * kFragment);
    };
    auto zeros_of = [&](int c) {
        return sp.vec + (unit0 + c - first) * Sizes::vec + kZeros * sizeof(float) + lane * 16;
    };
    auto load_t = [&](int c) {
        const char *at = sp.t + (unit0 + c - first) * Sizes::t + lane * 16;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int s = 0; s < 3; ++s)
                tf[p][s] = lower(at, zeros_of(c), p, s, 3);
    };
    auto load_pk = [&](int c) {
        const char *at = sp.p + (unit0 + c - first) * Sizes::p + lane * 16;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int s = 0; s < PP; ++s)
                pf[p][s] = lower(at, zeros_of(c), p, s, PP);
        at = sp.kt + (key_unit0 + c - first) * Sizes::kt + lane * 16;
#pragma unroll
        for (int x = 0; x < TW; ++x) {
            const int tile = w * TW + x < TILES ? w * TW + x : TILES - 1;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int s = 0; s < KP; ++s)
                    ktf[x][p][s] = *(const v8b *)(at + (size_t)((tile * 2 + p) * KP + s) * kFragment);
        }
    };
    if (first < last) {
        load_rows(first);
        load_vec(first);
        load_t(first);
        load_pk(first);
        publish();
        lds_barrier();
    }
    for (int c = first; c < last; ++c) {
        const int next = c + 1 < last ? c + 1 : c, start = kChunk * c;
        // K S and Q S, and what the corrections solve for
        v4f x[3] = {}, y[PP] = {};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const v8b s = Sf[kb][p][lane];
#pragma unroll
                for (int e = 0; e < KP; ++e) {
                    if (e + p <= 2)
                        x[p] = mfma(kf[kb][e], s, x[p]);
                    if (e + p <= LAST)
                        y[p] = mfma(qf[kb][e], s, y[p]);
                }
            }
        float R[4], vr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            vr[r] = T::load(v[r]);
        const v4f Y = PP == 3 ? (y[PP - 1] + y[1]) + y[0] : y[1] + y[0];
        const v4f X = (x[2] + x[1]) + x[0];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            R[r] = start + out_row + r < n ? vr[r] - dk_row[r] * X[r] : 0.0f;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            v4b out;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                out[r] = next_plane(R[r]);
            ((v4b *)&Rf[w / 2][p][lane])[w % 2] = out;
        }
        load_rows(next);
        lds_barrier();
        // the corrections
        v4f u[3] = {};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                const v8b r = Rf[p][s][lane];
#pragma unroll
                for (int e = 0; e + s <= 2; ++e)
                    u[e + s] = mfma(tf[p][e], r, u[e + s]);
            }
        const v4f U = (u[2] + u[1]) + u[0];
        load_t(next);
        {
            v4f rest = U, scaled;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                scaled[r] = U[r] * w_row[r];
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                v4b out;
                if (p < PP) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        out[r] = next_plane(((float *)&rest)[r]);
                    ((v4b *)&Uf[w / 2][p < PP ? p : 0][lane])[w % 2] = out;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    out[r] = next_plane(((float *)&scaled)[r]);
                ((v4b *)&Wf[w / 2][p][lane])[w % 2] = out;
            }
        }
        lds_barrier();
        // the outputs and the state
        v4f o[PP] = {}, d[TW][3] = {};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                const v8b f = Wf[p][s][lane];
#pragma unroll
                for (int t = 0; t < TW; ++t)
#pragma unroll
                    for (int e = 0; e < KP; ++e)
                        if (e + s <= 2)
                            d[t][s] = mfma(ktf[t][p][e], f, d[t][s]);
            }
#pragma unroll
            for (int s = 0; s < PP; ++s) {
                const v8b f = Uf[p][s][lane];
#pragma unroll
                for (int e = 0; e + s <= LAST; ++e)
                    o[e + s] = mfma(pf[p][e], f, o[e + s]);
            }
        }
#pragma unroll
        for (int t = 0; t < TW; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[t][r] = __builtin_fmaf(D, S[t][r], (d[t][2][r] + d[t][1][r]) + d[t][0][r]);
        publish();
        const v4f O = PP == 3 ? (o[PP - 1] + o[1]) + o[0] : o[1] + o[0];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = start + out_row + r;
            if (in && t < n)
                o_at[t * a.d.o_step_stride] = T::store(__builtin_fmaf(dq_row[r], Y[r], O[r]));
        }
        load_pk(next);
        load_vec(next);
        lds_barrier();
    }
    // steps behind the last one of this span: zeros
    const int from = n > kChunk * first ? n : kChunk * first;
    const int64_t to = (int64_t)kChunk * (first + (int64_t)sp.count);
    const int until = to < steps ? (int)to : steps;
    if (in)
        for (int t = from + tid / 16; t < until; t += 16)
            o_at[t * a.d.o_step_stride] = 0;
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int at = row_of(w * TW + x, 4 * g + r);
            if (sp.to && in && at < dk)
                sp.to[state_at + (int64_t)at * dv] = S[x][r];
        }
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
// last-level cache, where the second kernel finds them).
constexpr size_t kMostWorkspace = (size_t)256 << 20;
template <class T, int KB> static uint64_t span_of(const rnn_delta_desc &d, bool direct)
{
    const uint64_t all = chunks_of(d), most = kMostWorkspace / layout_of<T, KB>(d, 1, direct).all;
    return most < 1 ? 1 : most < all ? most : all;
}

template <class T, int KB, bool DIRECT> static int chunks_go(const DeltaArgs &a, hipStream_t s)
{
    const uint64_t all = chunks_of(a.d), span = span_of<T, KB>(a.d, DIRECT);
    const DeltaLayout l = layout_of<T, KB>(a.d, span, DIRECT);
    const uint64_t rounds = ((uint64_t)a.d.batch * a.d.heads + 7) / 8;
    const uint64_t slices = ((uint64_t)a.d.value_dim + 15) / 16;
    if (!launchable(rounds * 8 * span, 256) || !launchable(rounds * 8 * slices, 256))
        return (int)hipErrorInvalidConfiguration;
    char *ws = (char *)a.workspace;
    float *between = a.state_out ? a.state_out : span < all ? (float *)(ws + l.states) : nullptr;
    for (uint64_t first = 0; first < all; first += span) {
        const uint64_t count = all - first < span ? all - first : span;
        const DeltaSpan sp{(uint32_t)first, (uint32_t)count, ws + l.t, ws + l.p, ws + l.vec, ws + l.kt,
                           ws + l.packed, first == 0 ? a.state_in : between, between};
        delta_prepare_kernel<T, KB, DIRECT>
            <<<dim3((uint32_t)(rounds * 8 * count)), dim3(256), 0, s>>>(a, sp);
        int rc = (int)hipGetLastError();
        if (rc)
            return rc;
        delta_chunks_kernel<T, KB, DIRECT>
            <<<dim3((uint32_t)(rounds * 8 * slices)), dim3(256), 0, s>>>(a, sp, (uint32_t)slices);
        rc = (int)hipGetLastError();
        if (rc)
            return rc;
    }
    return 0;
}

// f(type, blocks of 32 rows of the state, whether keys and queries are operands as
// they are)
template <class F> static auto with_sizes(const rnn_delta_desc &d, F &&f)
{
    auto blocks = [&](auto type) {
        using T = decltype(type);
        auto at = [&](auto kb) {
            constexpr int KB = decltype(kb)::value;
            if constexpr (std::is_same<T, BF16>::value)
                if (d.key_dim == 32 * KB)
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
