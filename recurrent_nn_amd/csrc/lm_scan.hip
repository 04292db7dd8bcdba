// lm_scan.hip -- selective state space scan.
//
//   s = softplus(dt + dt_bias);  h[n] = exp(s A[n]) h[n] + s x B[n]
//   y = (sum_n C[n] h[n] + D x) silu(z)
//
// Bound by the vector unit: a state's step is three products, one exp2 and two
// additions (24 issue cycles a wave, exp2 is 8 of them), against 8 to 16 bytes
// a channel's step.  So each exp is computed once, every instruction of the
// inner loop works on states, and all else (loads, softplus, conversions,
// skip, gate, stores) is done by other waves of the workgroup.
#include <type_traits>

#include "lm_common.h"

namespace rnnamd {

// log(1 + exp(v)) = max(v, 0) + log1p(w), w = exp(-|v|) in (0, 1].  With
// q = w / (2 + w), log1p(w) = 2 atanh(q) = 2 q (1 + q^2/3 + q^4/5 + ...): no
// cancellation for small w; q <= 1/3, so seven terms reach 2^-26.  (NaN goes
// through w, infinities through the maximum.)
__device__ __forceinline__ float softplus(float v)
{
    const float w = __builtin_amdgcn_exp2f(-__builtin_fabsf(v) * kLog2e);
    const float q = w * __builtin_amdgcn_rcpf(2.0f + w);
    const float r = q * q;
    float p = 1.0f / 13.0f;
    p = __builtin_fmaf(p, r, 1.0f / 11.0f);
    p = __builtin_fmaf(p, r, 1.0f / 9.0f);
    p = __builtin_fmaf(p, r, 1.0f / 7.0f);
    p = __builtin_fmaf(p, r, 1.0f / 5.0f);
    p = __builtin_fmaf(p, r, 1.0f / 3.0f);
    p = __builtin_fmaf(p, r, 1.0f);
    return __builtin_fmaf(q + q, p, __builtin_fmaxf(v, 0.0f));
}

__device__ __forceinline__ int64_t row_length(const int32_t *lens, int64_t b, int64_t steps)
{
    if (!lens)
        return steps;
    const int64_t l = lens[b];
    return l < 0 ? 0 : (l < steps ? l : steps);
}

// Cross-lane moves within a row of 16 lanes, which the compiler folds into the
// instruction that uses them.
template <int CTRL> __device__ __forceinline__ float lanes(float v)
{
    return __uint_as_float(__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
constexpr int kBroadcast = 0x150;      // + i: lane i of the row to all its lanes
constexpr int kXor1 = 0xB1;            // quad_perm [1,0,3,2]
constexpr int kXor2 = 0x4E;            // quad_perm [2,3,0,1]
constexpr int kHalfMirror = 0x141;     // lane i from lane 7 - i of its 8
constexpr int kRor8 = 0x128;           // lane i from lane i xor 8 of its 16

// 16 values a lane, summed over the 16 lanes of a row: lane i gets the sum of
// value i.  Each stage adds across one bit of the lane number and keeps, in
// each lane, the half of the values that the lane will end with: 33
// instructions where 16 full sums take 64.  The first two stages select with
// the bank mask of the addition itself (a bank is four lanes).  The wait
// states before a cross-lane read of a fresh register are inside the blocks.
__device__ __forceinline__ float row_sums(const float (&p)[16], int lane)
{
    float r[8], q[4];
#define RNN_ADD2(out, a, b, perm, mask)                                                     \
    "v_add_f32_dpp " out ", " a ", " a " " perm " row_mask:0xf bank_mask:0xf\n\t"           \
    "v_add_f32_dpp " out ", " b ", " b " " perm " row_mask:0xf bank_mask:" mask "\n\t"
#pragma unroll
    for (int k = 0; k < 8; k += 4)
        asm("s_nop 1\n\t"
            RNN_ADD2("%0", "%4", "%8", "row_ror:8", "0xc")
            RNN_ADD2("%1", "%5", "%9", "row_ror:8", "0xc")
            RNN_ADD2("%2", "%6", "%10", "row_ror:8", "0xc")
            RNN_ADD2("%3", "%7", "%11", "row_ror:8", "0xc")
            : "=&v"(r[k]), "=&v"(r[k + 1]), "=&v"(r[k + 2]), "=&v"(r[k + 3])
            : "v"(p[k]), "v"(p[k + 1]), "v"(p[k + 2]), "v"(p[k + 3]), "v"(p[k + 8]),
              "v"(p[k + 9]), "v"(p[k + 10]), "v"(p[k + 11]));
    asm("s_nop 1\n\t"
        RNN_ADD2("%0", "%4", "%8", "row_half_mirror", "0xa")
        RNN_ADD2("%1", "%5", "%9", "row_half_mirror", "0xa")
        RNN_ADD2("%2", "%6", "%10", "row_half_mirror", "0xa")
        RNN_ADD2("%3", "%7", "%11", "row_half_mirror", "0xa")
        : "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3])
        : "v"(r[0]), "v"(r[1]), "v"(r[2]), "v"(r[3]), "v"(r[4]), "v"(r[5]), "v"(r[6]), "v"(r[7]));
#undef RNN_ADD2
    const bool b1 = lane & 2, b0 = lane & 1;
    const float u = (b1 ? q[2] : q[0]) + lanes<kXor2>(b1 ? q[0] : q[2]);
    const float w = (b1 ? q[3] : q[1]) + lanes<kXor2>(b1 ? q[1] : q[3]);
    return (b0 ? w : u) + lanes<kXor1>(b0 ? u : w);
}

// Sum over groups of L lanes, in every lane of the group.
template <int L> __device__ __forceinline__ float group_sum(float v)
{
    if (L > 1)
        v += lanes<kXor1>(v);
    if (L > 2)
        v += lanes<kXor2>(v);
    if (L > 4)
        v += lanes<kHalfMirror>(v);
    if (L > 8)
        v += lanes<kRor8>(v);
    return v;
}

// ---------------------------------------------------------------------------
// A few steps (single tokens): bound by the states, read and written once.
// A lane holds four states, L lanes a channel; 16-byte accesses where the
// states divide by four.  64 tokens x 4096 x 16: 8.6 us, 4.2 TB/s.
// ---------------------------------------------------------------------------

// FOURS: the states divide by four, so that a lane's are one load.
template <class T, int L, bool FOURS>
__global__ __launch_bounds__(256) void scan_steps_kernel(ScanArgs a, uint32_t row_blocks,
                                                        uint32_t per)
{
    using raw = typename T::raw;
    const int64_t b = blockIdx.x / row_blocks;
    const int64_t c = (blockIdx.x % row_blocks * 256ull + threadIdx.x) / L;
    const int n0 = threadIdx.x % L * 4;
    const int64_t steps = a.d.steps, len = row_length(a.lens, b, steps);
    const int N = (int)a.d.states;
    // (with FOURS a lane has four states or none)
    if (c >= a.d.dim)
        return;
    const bool mine = n0 < N;
    auto real = [&](int i) { return FOURS ? mine : n0 + i < N; };
    const int64_t at = (b * a.d.dim + c) * N + n0;
    const uint32_t g = (uint32_t)c / per;       // per: channels of a group of B and C
    // (no load depends on a condition: it would be waited for on the spot)
    const int n_load = mine ? n0 : 0;
    const float *A_at = a.A + c * N + n_load;
    const float *h_at = a.state_in ? a.state_in + (b * a.d.dim + c) * N + n_load : A_at;
    float h[4], A[4];
    if (FOURS) {
        __builtin_memcpy(h, __builtin_assume_aligned(h_at, 4), 16);
        __builtin_memcpy(A, __builtin_assume_aligned(A_at, 4), 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + i < N ? n0 + i - n_load : 0;
            h[i] = h_at[n];
            A[i] = A_at[n];
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f;
    const float D = a.D ? a.D[c] : 0.0f;
    const raw *x = (const raw *)a.x + b * a.d.x_batch_stride + c;
    const raw *dt = (const raw *)a.dt + b * a.d.dt_batch_stride + c;
    // without a gate x is loaded in its place, and not used
    const raw *z = a.z ? (const raw *)a.z + b * a.d.z_batch_stride + c : x;
    const int64_t z_step = a.z ? a.d.z_step_stride : a.d.x_step_stride;
    const raw *B = (const raw *)a.B + b * a.d.B_batch_stride + g * a.d.B_group_stride + n_load;
    const raw *C = (const raw *)a.C + b * a.d.C_batch_stride + g * a.d.C_group_stride + n_load;
    raw *y = (raw *)a.y + b * a.d.y_batch_stride + c;
    if (!a.state_in)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = 0.0f;
    for (int64_t t = 0; t < len; ++t) {
        Words4<T> Bw, Cw;
        if (FOURS) {
            Bw.load(B + t * a.d.B_step_stride);
            Cw.load(C + t * a.d.C_step_stride);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + i < N ? n0 + i - n_load : 0;
                Bw.set(i, B[t * a.d.B_step_stride + n]);
                Cw.set(i, C[t * a.d.C_step_stride + n]);
            }
        }
        const float xv = T::load(x[t * a.d.x_step_stride]);
        const raw zv = z[t * z_step];
        float s = T::load(dt[t * a.d.dt_step_stride]) + bias;
        if (a.d.dt_softplus)
            s = softplus(s);
        const float sx = s * xv;
        float p = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (real(i)) {
                h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(s * (A[i] * kLog2e)), h[i],
                                      sx * Bw.get(i));
                p = __builtin_fmaf(Cw.get(i), h[i], p);
            }
        p = group_sum<L>(p);
        if (a.D)
            p = __builtin_fmaf(D, xv, p);
        if (a.z)
            p *= silu(T::load(zv));
        if (n0 == 0)
            y[t * a.d.y_step_stride] = T::store(p);
    }
    if (n0 == 0)
        for (int64_t t = len; t < steps; ++t)
            y[t * a.d.y_step_stride] = T::store(0.0f);
    if (!a.state_out)
        return;
    if (FOURS && mine)
        __builtin_memcpy(__builtin_assume_aligned(a.state_out + at, 4), h, 16);
    if (!FOURS)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 + i < N)
                a.state_out[at + i] = h[i];
}

// ---------------------------------------------------------------------------
// Many steps
//
// A workgroup takes 16 channels of one batch row and walks a span of steps in
// tiles.  Four waves hold the states: a row of 16 lanes is one channel, lane
// i has the states i, i + 16, ... (S of them), so that step sizes come by a
// broadcast within the row that costs nothing, and sums over the states stay
// within it.  Four other waves prepare the next tile in LDS (step sizes s, s x,
// B and C in float32, the sums started with D x), and finish the last one
// (gate, rounding, store); the loads of the tile after next are in flight
// meanwhile.  One barrier a tile.
//
// With too few channels to fill the chip the steps are cut into spans:
// a first launch finds each span's state from zero and its sum of step sizes,
// the second starts each span from what the spans before it left,
//   h := exp(A sum s) h + h_span,  span by span,
// and has all the outputs.
//
// 8192 steps x 4096 channels x 16 states in bf16: 191 us once the clock has settled
// (216 to 235 in the first 20 ms from idle).  The vector unit is
// busy 78% of the time, with ten instructions a step (of four channels): five on
// the states, two for the sums, three of the preparing waves.  That is one
// workgroup a compute unit; splitting the steps instead would compute e and u
// twice.
// ---------------------------------------------------------------------------

struct Spans {
    uint32_t per;           // channels of a group of B and C
    uint32_t per16;         // its workgroups of 16 channels
    uint32_t groups16;      // all workgroups of a batch row
    uint32_t count;         // spans of a row
    int64_t length;         // steps of one, a multiple of the tile
    float *state;           // [batch, count + 1, dim, states]: each span's own, then state_in
    float *sum;             // [batch, count, dim]
};

constexpr int kTile = 64;

// FOURS: 16 channels or more and four states or more, so that four adjacent ones
// are one load: a last workgroup of fewer channels begins earlier and stores its
// own only; the last states are loaded from the fourth last one on, and moved.
// Else elements beyond the last are loaded as the last.  (No load depends on a
// condition: it would be waited for on the spot.)  What a workgroup computes for
// the channels of the one before is dropped, whatever it found in a state that
// the other may have replaced.  PAD: the states may not be whole sixteens; lanes
// beyond them are left out of sums.
template <class T, int S, bool FOURS, bool PAD, bool OUT>
__global__ __launch_bounds__(512) void scan_kernel(ScanArgs a, Spans sp)
{
    using raw = typename T::raw;
    constexpr int TT = kTile;
    constexpr int SP = TT + 20;         // 4 x 4 channels of 16 steps over all banks
    constexpr int BP = TT + 4;          // 16 lanes' 16-byte reads over all banks
    __shared__ float sh_s[2][16 * SP], sh_sx[2][16 * SP], sh_y[OUT ? 3 : 1][16 * SP];
    __shared__ __attribute__((aligned(16))) float sh_B[2][16 * S * BP],
        sh_C[OUT ? 2 : 1][OUT ? 16 * S * BP : 1];

    // Workgroups go to the 8 XCDs in turn: each XCD gets a run of this order, in
    // which four workgroups of adjacent channels (their pieces of a row share
    // cache lines) follow each other, then the spans, then the batch rows, and
    // the rows of the next four channel groups from another row on: the long
    // rows of a ragged batch are then spread over XCDs and compute units.
    const uint32_t total = gridDim.x, xcd = blockIdx.x % 8, q8 = total / 8, r8 = total % 8;
    const uint32_t id = xcd * q8 + (xcd < r8 ? xcd : r8) + blockIdx.x / 8;
    const uint32_t batch = (uint32_t)a.d.batch, each4 = 4 * sp.count * batch;
    const uint32_t four = id / each4, left = sp.groups16 - 4 * four, wide = left < 4 ? left : 4;
    const uint32_t in = id % each4, row = in / wide / sp.count;
    const uint32_t channels = 4 * four + in % wide, span = in / wide % sp.count;
    const int64_t b = (row + (uint64_t)four * (batch / 2 + 1)) % batch;
    const uint32_t g = channels / sp.per16, part = channels % sp.per16;
    const int64_t own = (int64_t)g * sp.per + part * 16, c_end = (int64_t)(g + 1) * sp.per;
    const int64_t c0 = FOURS && own + 16 > c_end ? c_end - 16 : own;
    const int64_t steps = a.d.steps, dim = a.d.dim;
    const int N = (int)a.d.states;
    const int64_t len = row_length(a.lens, b, steps);
    const int64_t start = span * sp.length;
    const int64_t stop = start + sp.length < steps ? start + sp.length : steps;
    const int64_t end = stop < len ? stop : len;
    const uint32_t tiles = end > start ? (uint32_t)((end - start + TT - 1) / TT) : 0;

    if (threadIdx.x >= 256) {
        // ---- prepare and finish: thread p has step p / 4 of a tile, channels (and
        // states, of each sixteen) 4 (p % 4) to + 3
        using P4 = Words4<T>;
        const int p = threadIdx.x - 256, ch = p % 4 * 4, t0 = p / 4;
        const int64_t c = c0 + ch;
        auto channel = [&](int v) { return FOURS || c + v < c_end ? c + v : c_end - 1; };
        float bias[4], D[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            bias[v] = a.dt_bias ? a.dt_bias[channel(v)] : 0.0f;
            D[v] = OUT && a.D ? a.D[channel(v)] : 0.0f;
        }
        // Rows of the thread's step in the tile that is loaded next, beyond the end
        // the last one's.
        struct Row {
            const raw *at;
            int64_t step;
            __device__ __forceinline__ void go(int64_t steps) { at += steps * step; }
        };
        Row x{(const raw *)a.x + b * a.d.x_batch_stride, a.d.x_step_stride};
        Row dt{(const raw *)a.dt + b * a.d.dt_batch_stride, a.d.dt_step_stride};
        // without a gate x is loaded in its place, and not used
        Row z = a.z ? Row{(const raw *)a.z + b * a.d.z_batch_stride, a.d.z_step_stride} : x;
        Row B{(const raw *)a.B + b * a.d.B_batch_stride + g * a.d.B_group_stride, a.d.B_step_stride};
        Row C{(const raw *)a.C + b * a.d.C_batch_stride + g * a.d.C_group_stride, a.d.C_step_stride};
        raw *y = (raw *)a.y + b * a.d.y_batch_stride + (start + t0) * a.d.y_step_stride + c;
        const int64_t t_first = start + t0 < end ? start + t0 : end - 1;
        x.go(t_first), dt.go(t_first), z.go(t_first), B.go(t_first), C.go(t_first);
        // from tile k to the next: a whole tile of steps, fewer before the end
        auto beyond = [&](uint32_t k) { return start + (int64_t)(k + 2) * TT > end; };
        auto to_next = [&](uint32_t k) {
            const int64_t now = start + (int64_t)k * TT + t0, next = now + TT;
            return (next < end ? next : end - 1) - (now < end ? now : end - 1);
        };
        P4 xr, dr, zr{}, Br[S], Cr[S];

        auto four_channels = [&](const raw *row) {
            P4 f;
            if (FOURS) {
                f.load(row + c);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    f.set(v, row[channel(v)]);
            }
            return f;
        };
        auto four_states = [&](const raw *row, int s) {
            P4 f;
            if (FOURS) {
                f.load(row + (!PAD || 16 * s + ch <= N - 4 ? 16 * s + ch : N - 4));
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    f.set(v, row[16 * s + ch + v < N ? 16 * s + ch + v : N - 1]);
            }
            return f;
        };
        auto load = [&](uint32_t k) {
            xr = four_channels(x.at);
            dr = four_channels(dt.at);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                Br[s] = four_states(B.at, s);
                if (OUT)
                    Cr[s] = four_states(C.at, s);
            }
            if (!beyond(k)) {
                x.go(TT), dt.go(TT), B.go(TT), C.go(TT);
            } else {
                const int64_t n = to_next(k);
                x.go(n), dt.go(n), B.go(n), C.go(n);
            }
        };
        auto prepare = [&](uint32_t k) {
            if (FOURS && PAD)
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    const int by = 16 * n + ch - (N - 4);
                    Br[n].drop(by);
                    if (OUT)
                        Cr[n].drop(by);
                }
            float s[4];
#pragma unroll
            for (int v = 0; v < 4; ++v)
                s[v] = dr.get(v) + bias[v];
            if (a.d.dt_softplus)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    s[v] = softplus(s[v]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int at = (ch + v) * SP + t0;
                const float xv = xr.get(v);
                sh_s[k % 2][at] = s[v];
                sh_sx[k % 2][at] = s[v] * xv;
                if (OUT)
                    sh_y[k % 3][at] = a.D ? D[v] * xv : 0.0f;
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    sh_B[k % 2][(ch + v + 16 * n) * BP + t0] = Br[n].get(v);
                    if (OUT)
                        sh_C[k % 2][(ch + v + 16 * n) * BP + t0] = Cr[n].get(v);
                }
            }
        };
        auto load_gate = [&](uint32_t k) {
            if (!OUT)
                return;
            zr = four_channels(z.at);
            z.go(!beyond(k) ? TT : to_next(k));
        };
        auto finish = [&](uint32_t k) {
            if (!OUT)
                return;
            float f[4];
            Pack<T, 4> out;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                f[v] = sh_y[k % 3][(ch + v) * SP + t0];
            if (a.z)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    f[v] *= silu(zr.get(v));
#pragma unroll
            for (int v = 0; v < 4; ++v)
                out.v[v] = T::store(f[v]);
            if (start + (int64_t)k * TT + t0 < end) {
                if (FOURS && c >= own) {
                    store_pack<T, 4>(y, out);
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (c + v >= own && c + v < c_end)
                            y[v] = out.v[v];
                }
            }
            y += TT * a.d.y_step_stride;
        };
        if (tiles > 0) {
            load(0);
            prepare(0);
            load(1);
        }
        __syncthreads();
        for (uint32_t k = 0; k < tiles; ++k) {
            if (k + 1 < tiles)
                prepare(k + 1);
            load(k + 2);
            if (k > 0)
                finish(k - 1);
            load_gate(k);
            __syncthreads();
        }
        if (tiles > 0)
            finish(tiles - 1);
        raw *zeros = (raw *)a.y + b * a.d.y_batch_stride + c;
        if (OUT)
            for (int64_t t = (end > start ? end : start) + t0; t < stop; t += 64)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (c + v >= own && c + v < c_end)
                        zeros[t * a.d.y_step_stride + v] = T::store(0.0f);
        return;
    }

    // ---- the states
    const int lane = threadIdx.x % 16, ch = threadIdx.x / 16;
    const int64_t c = c0 + ch;
    const bool on = c < c_end, stored = on && c >= own;
    float h[S], A[S], sums = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int n = lane + 16 * s;
        h[s] = A[s] = 0.0f;
        if (!on || (PAD && n >= N))
            continue;
        const float rate = len > 0 ? a.A[c * N + n] : 0.0f;
        if (sp.count > 1) {
            float *mine = sp.state + (b * (sp.count + 1) * dim + c) * N + n;
            float *first = mine + (int64_t)sp.count * dim * N;
            if (span == 0)
                h[s] = OUT ? *first : a.state_in ? a.state_in[(b * dim + c) * N + n] : 0.0f;
            if (!OUT && span == 0 && stored)
                *first = h[s];
            if (OUT && span > 0 && tiles > 0)
#pragma unroll 8
                for (uint32_t k = 0; k < span; ++k) {
                    const float own = mine[(int64_t)k * dim * N];
                    const float sum = sp.sum[(b * sp.count + k) * dim + c];
                    // the first span started from state_in
                    h[s] = k == 0 ? own
                                  : __builtin_fmaf(__builtin_amdgcn_exp2f(sum * (rate * kLog2e)),
                                                   h[s], own);
                }
        } else if (a.state_in) {
            h[s] = a.state_in[(b * dim + c) * N + n];
        }
        A[s] = rate * kLog2e;
    }
    const bool last_on = !PAD || lane + 16 * (S - 1) < N;

    // 16 steps from t of tile k; TAIL: only `left` of them count.
    auto block = [&](uint32_t k, int t, auto tail, int left) {
        constexpr bool TAIL = decltype(tail)::value;
        const float sv = sh_s[k % 2][ch * SP + t + lane];
        const float xv = sh_sx[k % 2][ch * SP + t + lane];
        if (!OUT)
            sums += !TAIL || lane < left ? sv : 0.0f;
        float p[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float Bq[S][4], Cq[S][4];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                __builtin_memcpy(Bq[s], __builtin_assume_aligned(
                                            &sh_B[k % 2][(lane + 16 * s) * BP + t + 4 * j], 16), 16);
                if (OUT)
                    __builtin_memcpy(Cq[s], __builtin_assume_aligned(
                                                &sh_C[k % 2][(lane + 16 * s) * BP + t + 4 * j], 16), 16);
            }
            auto one = [&](auto step) {
                constexpr int I = decltype(step)::value;
                const float sb = lanes<kBroadcast + I>(sv), xb = lanes<kBroadcast + I>(xv);
                float sum = 0.0f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float e = __builtin_amdgcn_exp2f(sb * A[s]);
                    const float next = __builtin_fmaf(e, h[s], xb * Bq[s][I % 4]);
                    h[s] = !TAIL || I < left ? next : h[s];
                    if (OUT) {
                        const float v = s == 0 ? Cq[s][I % 4] * h[s]
                                               : __builtin_fmaf(Cq[s][I % 4], h[s], sum);
                        sum = PAD && s == S - 1 && !last_on ? sum : v;
                    }
                }
                p[I] = sum;
            };
            if (j == 0) {
                one(std::integral_constant<int, 0>{}), one(std::integral_constant<int, 1>{});
                one(std::integral_constant<int, 2>{}), one(std::integral_constant<int, 3>{});
            } else if (j == 1) {
                one(std::integral_constant<int, 4>{}), one(std::integral_constant<int, 5>{});
                one(std::integral_constant<int, 6>{}), one(std::integral_constant<int, 7>{});
            } else if (j == 2) {
                one(std::integral_constant<int, 8>{}), one(std::integral_constant<int, 9>{});
                one(std::integral_constant<int, 10>{}), one(std::integral_constant<int, 11>{});
            } else {
                one(std::integral_constant<int, 12>{}), one(std::integral_constant<int, 13>{});
                one(std::integral_constant<int, 14>{}), one(std::integral_constant<int, 15>{});
            }
        }
        if (OUT) {
            float *out = &sh_y[k % 3][ch * SP + t + lane];
            *out += row_sums(p, lane);
        }
    };

    __syncthreads();
    for (uint32_t k = 0; k < tiles; ++k) {
        const int64_t here = end - (start + (int64_t)k * TT);
        const int count = here < TT ? (int)here : TT;
        for (int t = 0; t + 16 <= count; t += 16)
            block(k, t, std::false_type{}, 16);
        if (count % 16)
            block(k, count / 16 * 16, std::true_type{}, count % 16);
        __syncthreads();
    }
    if (!OUT) {
        sums = group_sum<16>(sums);
        if (stored && lane == 0)
            sp.sum[(b * sp.count + span) * dim + c] = sums;
    }
    // The row's last span that has steps (the first one if none has) has its
    // final state.
    const bool final = OUT && (end == len ? (span == 0 || start < len) : false);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int n = lane + 16 * s;
        if (!stored || (PAD && n >= N))
            continue;
        if (!OUT)
            sp.state[((b * (sp.count + 1) + span) * dim + c) * N + n] = h[s];
        else if (final && a.state_out)
            a.state_out[(b * dim + c) * N + n] = h[s];
    }
}

// Spans of a call: one, unless there are too few workgroups to fill the chip.
// A second pass costs two thirds of the first again, so it pays from four
// spans up: with G workgroups of 16 channels, 512 / G spans where that is four
// or more and each has 128 steps or more (chains of loads start each span).
static void spans_of(const rnn_scan_desc &d, Spans &sp)
{
    sp.per = (uint32_t)(d.dim / d.groups);
    sp.per16 = (sp.per + 15) / 16;
    const int64_t groups16 = sp.per16 * d.groups;
    sp.groups16 = (uint32_t)groups16;
    sp.count = 1;
    sp.length = (d.steps + kTile - 1) / kTile * kTile;
    int64_t count = 512 / (groups16 * d.batch);
    if (count > d.steps / 128)
        count = d.steps / 128;
    if (count < 4)
        return;
    sp.length = ((d.steps + count - 1) / count + kTile - 1) / kTile * kTile;
    sp.count = (uint32_t)((d.steps + sp.length - 1) / sp.length);
}

size_t scan_workspace(const rnn_scan_desc &d)
{
    Spans sp{};
    spans_of(d, sp);
    if (sp.count == 1)
        return 0;
    return (size_t)d.batch * d.dim * ((sp.count + 1) * d.states + sp.count) * 4;
}

template <class T, int S, bool FOURS, bool PAD>
static int scan_passes(const ScanArgs &a, const Spans &sp, hipStream_t s)
{
    const dim3 grid((uint32_t)(sp.groups16 * sp.count * a.d.batch)), block(512);
    if (sp.count > 1) {
        scan_kernel<T, S, FOURS, PAD, false><<<grid, block, 0, s>>>(a, sp);
        const int rc = (int)hipGetLastError();
        if (rc)
            return rc;
    }
    scan_kernel<T, S, FOURS, PAD, true><<<grid, block, 0, s>>>(a, sp);
    return (int)hipGetLastError();
}

template <class T, int S> static int scan_go(const ScanArgs &a, const Spans &sp, hipStream_t s)
{
    if (sp.per < 16 || a.d.states < 4)
        return scan_passes<T, S, false, true>(a, sp, s);
    return a.d.states % 16 ? scan_passes<T, S, true, true>(a, sp, s)
                           : scan_passes<T, S, true, false>(a, sp, s);
}

// No steps: the state is handed on.
__global__ __launch_bounds__(256) void scan_no_steps_kernel(const float *in, float *out, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        out[i] = in ? in[i] : 0.0f;
}

static int no_steps_go(const ScanArgs &a, hipStream_t s)
{
    const int64_t n = a.d.batch * a.d.dim * a.d.states;
    if (!launchable((uint64_t)(n + 255) / 256, 256))
        return (int)hipErrorInvalidConfiguration;
    scan_no_steps_kernel<<<dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, s>>>(a.state_in, a.state_out, n);
    return (int)hipGetLastError();
}

template <class T, int L> static int steps_go(const ScanArgs &a, hipStream_t s)
{
    const uint32_t per = (uint32_t)(a.d.dim / a.d.groups);
    const int64_t row_blocks = (a.d.dim * L + 255) / 256;
    if (!launchable((uint64_t)(row_blocks * a.d.batch), 256))
        return (int)hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)(row_blocks * a.d.batch)), block(256);
    if (a.d.states % 4 == 0)
        scan_steps_kernel<T, L, true><<<grid, block, 0, s>>>(a, (uint32_t)row_blocks, per);
    else
        scan_steps_kernel<T, L, false><<<grid, block, 0, s>>>(a, (uint32_t)row_blocks, per);
    return (int)hipGetLastError();
}

// Steps up to which the states stay in scan_steps_kernel, by the workgroups that
// scan_kernel would have: it spends about 1.6 us of a compute unit on starting
// each, and with 2048 or more the other one's waves fill the chip.  States up to 8
// leave half of scan_kernel's lanes idle.  In bf16 (scan_kernel, scan_steps_kernel):
// 512 workgroups, 16 states, 12 steps 7.8, 7.8 us; 1024, 16 steps 9.8, 9.5 us;
// 2048, 32 steps 18.2, 16.2 us and 48 steps 20, 27 us; 16384, 32 steps 123, 71 us;
// 4096, 8 states, 64 steps 42, 37 us and 128 steps 59, 70 us.
static int64_t few_steps(const rnn_scan_desc &d, const Spans &sp)
{
    const int64_t workgroups = (int64_t)sp.groups16 * d.batch;
    if (workgroups < 1024)
        return 8;
    if (workgroups < 2048)
        return 16;
    return workgroups >= 4096 && d.states <= 8 ? 64 : 32;
}

template <class T> static int scan_type(const ScanArgs &a, hipStream_t s)
{
    Spans sp{};
    spans_of(a.d, sp);
    if (a.d.steps <= few_steps(a.d, sp)) {
        if (a.d.states <= 4)
            return steps_go<T, 1>(a, s);
        if (a.d.states <= 8)
            return steps_go<T, 2>(a, s);
        if (a.d.states <= 16)
            return steps_go<T, 4>(a, s);
        return a.d.states <= 32 ? steps_go<T, 8>(a, s) : steps_go<T, 16>(a, s);
    }
    // (the kernel has four times their number in 32 bits)
    if (!launchable((uint64_t)sp.groups16 * sp.count * a.d.batch, 512))
        return (int)hipErrorInvalidConfiguration;
    sp.state = (float *)a.workspace;
    sp.sum = sp.state + (size_t)a.d.batch * (sp.count + 1) * a.d.dim * a.d.states;
    switch ((a.d.states + 15) / 16) {
    case 1: return scan_go<T, 1>(a, sp, s);
    case 2: return scan_go<T, 2>(a, sp, s);
    case 3: return scan_go<T, 3>(a, sp, s);
    default: return scan_go<T, 4>(a, sp, s);
    }
}

int launch_scan(const ScanArgs &a, hipStream_t s)
{
    if (a.d.steps == 0)
        return no_steps_go(a, s);
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: return scan_type<F32>(a, s);
    case RNN_DTYPE_BF16: return scan_type<BF16>(a, s);
    default: return scan_type<F16>(a, s);
    }
}

}  // namespace rnnamd
