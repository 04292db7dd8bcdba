// lm_delta.hip -- gated delta rule, step by step, for single tokens and short
// calls.
//
//   S = e^a S;  u = b (v - S^T k);  S = S + k u^T;  o = scale S^T q
//
// A state's columns are independent of each other.  A wave keeps 32 of them, all
// rows, in registers: lane 8 g + c has columns 4 c to 4 c + 3 of a quarter of each
// 32 rows, so that a load covers whole 128-byte lines.  With D = e^a, k^T S and q^T S of
// the state before the step are summed together, one reduction over the groups a
// step:  u = b (v - D k^T S),  o = scale (D q^T S + (q . k) u),  S = D S + k u^T.
// Norms of q and k are factors of these sums, and come with the same reduction.
//
// A single token is bound by HBM: its state read once and written once.  64 tokens x
// 32 heads x 128 x 128, 270 MB, 62 us, 4.4 TB/s; all of a wave's rows are asked for
// before the first is used (16 KB a wave).  Each further step of a call is a chain
// through the reduction, 2.1 us.
#include "lm_delta.h"

namespace rnnamd {

// The sum of v over the wave's eight groups of eight lanes, in all of them.
__device__ __forceinline__ float over_groups(float v)
{
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x128, 0xF, 0xF,
                                                               true));      // lane xor 8
    auto both = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(both[0]) + __uint_as_float(both[1]);                // lane xor 16
    both = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(both[0]) + __uint_as_float(both[1]);             // lane xor 32
}

// NI rows a lane; FULL: key_dim is 8 NI, else rows beyond it are zeros.
template <class T, int NI, bool FULL>
__global__ __launch_bounds__(256) void delta_steps_kernel(DeltaArgs a, uint32_t tiles)
{
    using raw = typename T::raw;
    const uint32_t lane = threadIdx.x % 64, c = lane % 8, group = lane / 8;
    const uint64_t id = (uint64_t)blockIdx.x * 4 + threadIdx.x / 64;
    const uint64_t bh = id / tiles;
    const uint32_t heads = (uint32_t)a.d.heads;
    const int64_t b = (int64_t)(bh / heads), head = (int64_t)(bh % heads);
    if (b >= a.d.batch)
        return;
    const int dk = (int)a.d.key_dim, dv = (int)a.d.value_dim, row0 = (int)group * 4;
    const int tile = (int)(id % tiles) * 32, col = tile + 4 * (int)c;
    const bool whole = tile + 32 <= dv;         // the wave's columns are all there
    const int steps = (int)a.d.steps, n = delta_steps(a, b);
    const int64_t key_head = head / (heads / a.d.key_heads);

    float S[NI][4];
    // register i has row 32 (i / 4) + 4 group + i % 4: four loads cover 32 rows
    auto row_of = [&](int i) { return 32 * (i / 4) + row0 + i % 4; };
    const int64_t state_at = (int64_t)bh * dk * dv + col;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            S[i][j] = 0.0f;
        if (a.state_in && (FULL || row_of(i) < dk)) {
            const float *p = a.state_in + state_at + (int64_t)row_of(i) * dv;
            if (whole) {
                __builtin_memcpy(S[i], p, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < dv)
                        S[i][j] = p[j];
            }
        }
    }

    const raw *q_at = (const raw *)a.q + b * a.d.q_batch_stride + key_head * a.d.q_head_stride;
    const raw *k_at = (const raw *)a.k + b * a.d.k_batch_stride + key_head * a.d.k_head_stride;
    const raw *v_at = (const raw *)a.v + b * a.d.v_batch_stride + head * a.d.v_head_stride;
    raw *o_at = (raw *)a.o + b * a.d.o_batch_stride + head * a.d.o_head_stride;
    const int64_t beta_at = b * a.d.beta_batch_stride + head, g_at = b * a.d.g_batch_stride + head;
    const float A = a.A ? a.A[head] : 0.0f, bias = a.dt_bias ? a.dt_bias[head] : 0.0f;

    struct Step {
        Pack<T, NI> k, q;
        raw v[4];
        float beta, g;
    };
    auto rows = [&](const raw *p) {
        Pack<T, NI> r;
        if (FULL) {
#pragma unroll
            for (int i = 0; i < NI; i += 4)
                __builtin_memcpy(&r.v[i], p + row_of(i), 4 * sizeof(raw));
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const raw x = p[row_of(i) < dk ? row_of(i) : dk - 1];
                r.v[i] = row_of(i) < dk ? x : (raw)0;
            }
        }
        return r;
    };
    auto load = [&](int t) {
        Step s;
        s.k = rows(k_at + t * a.d.k_step_stride);
        s.q = rows(q_at + t * a.d.q_step_stride);
        const raw *p = v_at + t * a.d.v_step_stride;
        if (whole) {
            __builtin_memcpy(s.v, p + col, sizeof(s.v));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s.v[j] = p[col + j < dv ? col + j : dv - 1];
        }
        s.beta = gate_at<T>(a.beta, a.d.gate_dtype, beta_at + t * a.d.beta_step_stride);
        s.g = a.g ? gate_at<T>(a.g, a.d.gate_dtype, g_at + t * a.d.g_step_stride) : 0.0f;
        return s;
    };
    auto put = [&](int t, const float (&o)[4]) {
        raw *p = o_at + t * a.d.o_step_stride + col;
        raw r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r[j] = T::store(o[j]);
        if (whole) {
            __builtin_memcpy(p, r, sizeof(r));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < dv)
                    p[j] = r[j];
        }
    };

    if (n > 0) {
        Step next = load(0);
        for (int t = 0; t < n; ++t) {
            const Step s = next;
            next = load(t + 1 < n ? t + 1 : t);
            float ks[4] = {}, qs[4] = {}, kk = 0.0f, qk = 0.0f, qq = 0.0f, k[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const float q = T::load(s.q.v[i]);
                k[i] = T::load(s.k.v[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ks[j] = __builtin_fmaf(k[i], S[i][j], ks[j]);
                    qs[j] = __builtin_fmaf(q, S[i][j], qs[j]);
                }
                kk = __builtin_fmaf(k[i], k[i], kk);
                qk = __builtin_fmaf(q, k[i], qk);
                qq = __builtin_fmaf(q, q, qq);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ks[j] = over_groups(ks[j]);
                qs[j] = over_groups(qs[j]);
            }
            qk = over_groups(qk);
            if (a.d.normalize) {
                kk = over_groups(kk);
                qq = over_groups(qq);
            }
            const float rk = key_scale(kk, a.d.normalize);
            const float rq = key_scale(qq, a.d.normalize) * a.d.scale;
            const float D = a.g ? expf(log_decay(s.g, a.A != nullptr, A, bias)) : 1.0f;
            const float rate = rate_of(s.beta, a.d.beta_sigmoid);
            float u[4], o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u[j] = rate * (T::load(s.v[j]) - D * (rk * ks[j]));
                o[j] = rq * __builtin_fmaf(rk * qk, u[j], D * qs[j]);
                u[j] *= rk;
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    S[i][j] = __builtin_fmaf(k[i], u[j], D * S[i][j]);
            if (group == 0)
                put(t, o);
        }
    }
    const float none[4] = {};
    for (int t = n + (int)group; t < steps; t += 8)
        put(t, none);
    if (!a.state_out)
        return;
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (FULL || row_of(i) < dk) {
            float *p = a.state_out + state_at + (int64_t)row_of(i) * dv;
            if (whole) {
                __builtin_memcpy(p, S[i], 16);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < dv)
                        p[j] = S[i][j];
            }
        }
}

template <class T, int NI> static int steps_go(const DeltaArgs &a, hipStream_t s)
{
    const uint64_t tiles = ((uint64_t)a.d.value_dim + 31) / 32;
    const uint64_t blocks = ((uint64_t)a.d.batch * a.d.heads * tiles + 3) / 4;
    if (!launchable(blocks, 256))
        return (int)hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)blocks), block(256);
    if (a.d.key_dim == 8 * NI)
        delta_steps_kernel<T, NI, true><<<grid, block, 0, s>>>(a, (uint32_t)tiles);
    else
        delta_steps_kernel<T, NI, false><<<grid, block, 0, s>>>(a, (uint32_t)tiles);
    return (int)hipGetLastError();
}

template <class T> static int delta_go(const DeltaArgs &a, hipStream_t s)
{
    if (a.d.key_dim <= 32)
        return steps_go<T, 4>(a, s);
    if (a.d.key_dim <= 64)
        return steps_go<T, 8>(a, s);
    if (a.d.key_dim <= 96)
        return steps_go<T, 12>(a, s);
    if (a.d.key_dim <= 128)
        return steps_go<T, 16>(a, s);
    return a.d.key_dim <= 192 ? steps_go<T, 24>(a, s) : steps_go<T, 32>(a, s);
}

// Chunks from so many steps on, whatever the batch, so that a row alone gives the same
// bits as in a batch; and where the rows of a chunk lie within what 32 bits of a lane's
// address reach.  Steps against chunks, bf16, key and value dim 128: of one row of 32
// heads 8 steps 23 us against 17, 12 steps 31 and 17; of 16 rows 12 steps 52 and 70,
// 16 steps 65 and 71, 20 steps 78 and 72; of 64 rows 8 steps 144 and 257, 16 steps 245
// and 259, 24 steps 349 and 270.
static bool in_chunks(const rnn_delta_desc &d)
{
    const int64_t most = ((int64_t)1 << 31) / (64 * (d.dtype == RNN_DTYPE_F32 ? 4 : 2)) - 65536;
    return d.steps > 8 && d.q_step_stride < most && d.k_step_stride < most && d.v_step_stride < most &&
           d.o_step_stride < most && d.value_dim < 65536;
}

size_t delta_workspace(const rnn_delta_desc &d) { return in_chunks(d) ? delta_chunks_workspace(d) : 0; }

int launch_delta(const DeltaArgs &a, hipStream_t s)
{
    if (in_chunks(a.d))
        return launch_delta_chunks(a, s);
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: return delta_go<F32>(a, s);
    case RNN_DTYPE_BF16: return delta_go<BF16>(a, s);
    default: return delta_go<F16>(a, s);
    }
}

}  // namespace rnnamd
