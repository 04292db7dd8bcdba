// lm_scores.hip -- log probability of a given token, entropy, rank and the
// most likely alternatives of each row of logits.
//
//   S = sum exp(x - m),  W = sum exp(x - m) (x - m)
//   logprob = (x_token - m) - log S,  entropy = log S - W / S   (for any m)
//
// Bound by HBM: the logits are read once.  What a thread keeps beside S and W
// of its elements: the count that precedes the token, and the maxima of eight
// parts of them.  From the threads' maxima each wave takes the value that
// top / 4 of its lanes reach; the least of the four is a bound that at least
// `top` elements reach, so that only the parts that reach it are read again
// (a few more than `top`, from the caches), and what they hold above it is
// ordered.  Few rows are cut into segments, which a second launch joins.
// 1024 x 131072 in bf16: 58 us with 20 alternatives (4.6 TB/s), 53 with none.
#include <type_traits>

#include "lm_order.h"

namespace rnnamd {

constexpr float kLowest = -3.402823466e38f;
// Exponents below it count as it: exp is 0 there, and -inf (0 inf = NaN) stays out.
constexpr float kFar = -1000.0f;

// Sums relative to m.  The formulas hold for any m, but S of a row that is nearly
// certain is 1 and a little, W a little: relative to a lower m both are larger by
// e^(max - m), log S is near max - m, and what is left of its and W / S's rounding
// when they meet x - m is that of values near max - m (1.2e-6 for m up to 8 below).
// So m is the largest of what a wave has read, and only grows: no term of W is ever
// positive.
struct Sums {
    float m, sum, cross;
    __device__ __forceinline__ void rebase(float to)
    {
        const float d = __builtin_fmaxf(m - to, kFar);
        const float scale = __builtin_amdgcn_exp2f(d * kLog2e);
        cross = __builtin_fmaf(d, sum, cross) * scale;
        sum *= scale;
        m = to;
    }
    __device__ __forceinline__ void join(Sums o)
    {
        const float to = __builtin_fmaxf(m, o.m);
        rebase(to);
        o.rebase(to);
        sum += o.sum;
        cross += o.cross;
    }
};
struct Part {               // of a segment of a row
    Sums s;
    uint32_t before;
};

// The parts of a workgroup's 256 threads together, in every thread.
__device__ __forceinline__ Part over_workgroup(Part p, Part (&parts)[4])
{
    p.s.rebase(value_of(wave_max(value_key(p.s.m))));
    p.s.sum = wave_sum(p.s.sum);
    p.s.cross = wave_sum(p.s.cross);
    p.before = wave_sum(p.before);
    if (threadIdx.x % 64 == 0)
        parts[threadIdx.x / 64] = p;
    __syncthreads();
    Part all = parts[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
        all.s.m = __builtin_fmaxf(all.s.m, parts[i].s.m);
    all.s.sum = all.s.cross = 0.0f;
    all.before = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Part o = parts[i];
        o.s.rebase(all.s.m);
        all.s.sum += o.s.sum;
        all.s.cross += o.s.cross;
        all.before += o.before;
    }
    return all;
}

struct Token {
    int64_t id;
    bool known;
    float value;
};
template <class T> __device__ __forceinline__ Token token_of(const ScoresArgs &a, int64_t row,
                                                            const typename T::raw *x)
{
    Token t{-1, false, 0.0f};
    if (a.tokens)
        t.id = a.d.token_bytes == 8 ? ((const int64_t *)a.tokens)[row] : ((const int32_t *)a.tokens)[row];
    t.known = t.id >= 0 && t.id < a.d.vocab;
    if (t.known)
        t.value = T::load(x[t.id]);
    return t;
}

// A row's outputs from its sums and its ordered best keys.
__device__ __forceinline__ void put_scores(const ScoresArgs &a, int64_t row, const Part &p,
                                           const Token &t, const uint64_t *sorted, uint32_t kept)
{
    const float lse = __builtin_amdgcn_logf(p.s.sum) * kLn2;
    if (threadIdx.x == 0) {
        if (a.logprob)
            a.logprob[row] = t.known ? (t.value - p.s.m) - lse : __uint_as_float(0x7FC00000u);
        if (a.entropy)
            a.entropy[row] = lse - p.s.cross / p.s.sum;
        if (a.rank)
            a.rank[row] = t.known ? (int32_t)p.before : -1;
    }
    const int j = threadIdx.x;
    if (j < a.d.top) {
        const bool have = (uint32_t)j < kept;
        const uint64_t key = have ? sorted[j] : 0;
        if (a.top_logprobs)
            a.top_logprobs[row * a.d.top + j] =
                have ? (key_value(key) - p.s.m) - lse : -__builtin_inff();
        if (a.top_ids)
            a.top_ids[row * a.d.top + j] = have ? (int32_t)key_index(key) : -1;
    }
}

// One segment of a row: packs [first, last) of 8 elements.  A thread takes
// every 256th pack, U at a time: the loads of a batch are in flight while the
// one before is summed.  Where a row of 16-bit elements begins between two words
// (every other row of an odd vocabulary), packs begin with its second element,
// and the first one is taken by itself: 1024 x 131073 in bf16 60 us (70 without), no
// alternatives 53 (61).
template <class T> __global__ __launch_bounds__(256) void scores_kernel(ScoresArgs a,
                                                                      uint32_t segments,
                                                                      uint32_t segment_packs)
{
    using raw = typename T::raw;
    constexpr uint32_t PARTS = 8, U = sizeof(raw) == 2 ? 4 : 2, BATCH = 256 * U;
    constexpr int WORDS = 8 * sizeof(raw) / 4;
    __shared__ uint64_t list[kList], sorted[RNN_SCORES_MAX_TOP];
    __shared__ float most[PARTS][256];
    __shared__ uint32_t count, bounds[4];
    __shared__ uint16_t items[256];
    __shared__ Part parts[4];
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int64_t row = blockIdx.x / segments;
    const uint32_t segment = blockIdx.x % segments;
    const raw *row_at = (const raw *)a.logits + row * a.d.logits_stride;
    const uint32_t skip = sizeof(raw) == 2 && ((uintptr_t)row_at & 2) ? 1 : 0;
    const uint32_t V = (uint32_t)a.d.vocab - skip, all = (V + 7) / 8;
    const uint32_t first = segment * segment_packs;
    const uint32_t last = first + segment_packs < all ? first + segment_packs : all;
    const uint32_t whole = last < V / 8 ? last : V / 8;      // packs of all 8 elements end here
    const raw *x = row_at + skip;
    const bool head = skip && segment == 0;     // x[-1] is this segment's
    const uint32_t batches = whole > first ? (whole - first + BATCH - 1) / BATCH : 0;
    const uint32_t part_batches = (batches + PARTS - 1) / PARTS;

    uint32_t next[U][WORDS];
    auto load = [&](uint32_t batch) {           // beyond the end: the last pack again
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t i = first + batch * BATCH + u * 256 + tid;
            __builtin_memcpy(next[u], x + 8 * (int64_t)(i < whole ? i : whole - 1), sizeof(next[u]));
        }
    };
    if (batches > 0)
        load(0);

    const Token tk = token_of<T>(a, row, row_at);
    const float mine = tk.value;
    const int64_t id = tk.id - skip;            // in x; the row's first element may be -1
    // What counts as before the token: in packs before the token's own
    // !(x <= lower), lower the next value below it; from its own on
    // !(x <= mine).  The own pack's equal entries before it are added after.
    // (-inf is preceded by everything of lower index; a NaN is counted below.)
    const bool unordered = mine != mine;
    const uint32_t token_pack = tk.known && id > 0 ? (uint32_t)(id / 8) : 0;
    float lower = mine;
    {
        const uint32_t u = __float_as_uint(mine);
        lower = mine == 0.0f ? -__uint_as_float(1u)
                             : __uint_as_float((u & 0x80000000u) ? u + 1u : u - 1u);
        if (mine == -__builtin_inff())
            lower = __uint_as_float(0x7FC00000u);
    }

    Part p{{kLowest, 0.0f, 0.0f}, 0};
    uint32_t before = 0;                        // of the wave
    float top_of_part = -__builtin_inff(), top_of_all = top_of_part;
    auto one = [&](const float (&f)[8], float edge) {
        const float pm = __builtin_fmaxf(
            __builtin_fmaxf(__builtin_fmaxf(f[0], f[1]), __builtin_fmaxf(f[2], f[3])),
            __builtin_fmaxf(__builtin_fmaxf(f[4], f[5]), __builtin_fmaxf(f[6], f[7])));
        top_of_part = __builtin_fmaxf(top_of_part, pm);
        // a few times a row (1024 x 131072 that rise throughout: 58 us, 48 without)
        if (__builtin_expect(__ballot(pm > p.s.m) != 0, 0))
            p.s.rebase(value_of(wave_max(value_key(pm))));
        float e[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            const float d = f[v] - p.s.m;
            e[v] = __builtin_amdgcn_exp2f(d * kLog2e);
            p.s.cross = __builtin_fmaf(e[v], __builtin_fmaxf(d, kFar), p.s.cross);
            before += __popcll(__ballot(!(f[v] <= edge)));
        }
        p.s.sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    };
    uint32_t in_part = 0, part = 0;
    // a batch; LAST: the last one, whose packs may lie beyond the end
    auto sum_batch = [&](uint32_t b, auto last_one) {
        constexpr bool LAST = decltype(last_one)::value;
        uint32_t now[U][WORDS];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u)
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
                now[u][w] = next[u][w];
        if (!LAST)
            load(b + 1);
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t i = first + b * BATCH + u * 256 + tid;
            const bool beyond = LAST && i >= whole;
            float f[8];
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                if constexpr (sizeof(raw) == 4)
                    f[v] = T::load(now[u][v]);
                else
                    f[v] = T::load((raw)(v % 2 ? now[u][v / 2] >> 16 : now[u][v / 2] & 0xFFFFu));
            }
            if (LAST)
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    f[v] = beyond ? -__builtin_inff() : f[v];
            // (what lies beyond must not count as before a token)
            one(f, !beyond && i < token_pack ? lower : mine);
        }
        if (++in_part == part_batches || LAST) {
            most[part][tid] = top_of_part;
            top_of_all = __builtin_fmaxf(top_of_all, top_of_part);
            top_of_part = -__builtin_inff();
            in_part = 0;
            ++part;
            if (LAST)
                for (; part < PARTS; ++part)
                    most[part][tid] = -__builtin_inff();
        }
    };
    for (uint32_t b = 0; b + 1 < batches; ++b)
        sum_batch(b, std::false_type{});
    if (batches > 0)
        sum_batch(batches - 1, std::true_type{});
    // the last elements, fewer than a pack, one a thread
    const uint32_t rest = last * 8 > V ? V - whole * 8 : 0;
    const float f_rest = tid < rest ? T::load(x[whole * 8 + tid]) : -__builtin_inff();
    if (wave == 0 && rest > 0) {
        float f[8];
#pragma unroll
        for (int v = 1; v < 8; ++v)
            f[v] = -__builtin_inff();
        f[0] = f_rest;
        one(f, mine);
        top_of_all = __builtin_fmaxf(top_of_all, f_rest);
    }
    const float f_head = head && tid == 0 ? T::load(x[-1]) : -__builtin_inff();
    if (wave == 0 && head) {
        float f[8];
#pragma unroll
        for (int v = 1; v < 8; ++v)
            f[v] = -__builtin_inff();
        f[0] = f_head;
        one(f, __builtin_inff());
        top_of_all = __builtin_fmaxf(top_of_all, f_head);
    }
    if (lane == 0)
        p.before = before;
    if (tid == 0 && tk.known && token_pack >= first && token_pack < last)
        for (int64_t v = token_pack * 8; v < id; ++v)
            p.before += T::load(x[v]) == mine;
    if (tid == 0 && head && tk.known && id >= 0)
        p.before += !(f_head <= lower);
    p = over_workgroup(p, parts);
    const bool odd = !(p.s.sum < __builtin_inff());     // NaN or infinite entries
    if (tk.known && (odd || unordered)) {               // count by the keys themselves
        const uint64_t mine_key = order_key(mine, (uint32_t)tk.id);
        Part q{{kLowest, 0.0f, 0.0f}, 0};
        for (uint32_t v = first * 8 + tid; v < V && v < last * 8; v += 256)
            q.before += order_key(T::load(x[v]), v + skip) > mine_key;
        if (tid == 0 && head)
            q.before += order_key(f_head, 0) > mine_key;
        __syncthreads();
        p.before = over_workgroup(q, parts).before;
    }

    const int top = a.d.top;
    Best best;
    best.begin(list, sorted, &count, top);
    if (top > 0) {
        // The bound, to 16 bits: the largest t that enough lanes reach.
        const uint32_t key = value_key(top_of_all), enough = (top + 3) / 4;
        uint32_t t = 0;
        for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit /= 2)
            if (__popcll(__ballot(key >= (t | bit))) >= (int)enough)
                t |= bit;
        if (lane == 0)
            bounds[wave] = t;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t = bounds[i] < t ? bounds[i] : t;
        // (cut to 16 bits, -inf lies below every number's key)
        const float edge = t < value_key(kLowest) ? -__builtin_inff() : value_of(t);
        if (!odd && batches > 0)
            for (uint32_t s = 0; s < PARTS; ++s)
                if (most[s][tid] >= edge) {
                    const uint32_t at = atomicAdd(&count, 1u);
                    if (at < 256)
                        items[at] = (uint16_t)(s * 256 + tid);
                }
        uint32_t n = best.offered();
        best.forget();
        const bool few = !odd && n <= 256;
        const uint32_t item_packs = part_batches * U;
        const uint32_t packs = few ? n * item_packs : last - first;
        auto wanted = [&](float f) { return odd || f >= edge; };
        if (head)
            best.offer(order_key(f_head, 0), tid == 0 && wanted(f_head));
        if (few)
            best.offer(order_key(f_rest, skip + whole * 8 + tid), tid < rest && wanted(f_rest));
        best.settle(best.offered());
        for (uint32_t base = 0; base < packs; base += 256) {
            const uint32_t q = base + tid;
            bool on = q < packs;
            uint32_t i = first + q;
            if (few && on) {
                const uint32_t item = items[q / item_packs], r = q % item_packs;
                i = first + item / 256 * part_batches * BATCH + r * 256 + item % 256;
                on = i < whole;
            }
            Pack<T, 8> pk{};
            if (on)
                pk = logits_pack<T>(x, i, V);
            uint64_t keys[8];
            uint32_t want = 0;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const float f = T::load(pk.v[v]);
                keys[v] = order_key(f, skip + 8 * i + v);
                want |= (uint32_t)(on && 8 * i + v < V && wanted(f)) << v;
            }
            best.offer(keys, want);
            n = best.offered();
            if (n > kList) {            // too many at once: an eighth of them at a time
                best.forget();
#pragma unroll 1
                for (int v = 0; v < 8; ++v) {
                    const float f = T::load(pk.v[0]);
                    best.offer(order_key(f, skip + 8 * i + v), on && 8 * i + v < V && wanted(f));
                    best.order(best.offered());
#pragma unroll
                    for (int u = 0; u < 7; ++u)
                        pk.v[u] = pk.v[u + 1];
                }
            } else if (n > kList / 2) {
                best.order(n);
            } else {
                best.settle(n);
            }
        }
        best.order(best.offered());
    }
    if (segments == 1) {
        put_scores(a, row, p, tk, sorted, best.kept);
        return;
    }
    uint64_t *keys = (uint64_t *)a.workspace + (int64_t)blockIdx.x * top;
    Part *out = (Part *)((uint64_t *)a.workspace + (int64_t)gridDim.x * top) + blockIdx.x;
    if (tid == 0)
        *out = p;
    if (tid < (uint32_t)top)
        keys[tid] = tid < best.kept ? sorted[tid] : 0;
}

constexpr uint32_t kMostSegments = 512;

// The segments of a row together.
template <class T> __global__ __launch_bounds__(256) void scores_join_kernel(ScoresArgs a,
                                                                           uint32_t segments)
{
    __shared__ uint64_t list[kList], sorted[RNN_SCORES_MAX_TOP];
    __shared__ uint32_t count;
    __shared__ Part parts[4];
    const int64_t row = blockIdx.x;
    const uint32_t top = (uint32_t)a.d.top, n_keys = segments * top;
    const uint64_t *keys = (const uint64_t *)a.workspace + row * n_keys;
    const Part *in = (const Part *)((const uint64_t *)a.workspace + (int64_t)gridDim.x * n_keys) +
                     row * segments;
    const Token tk = token_of<T>(a, row, (const typename T::raw *)a.logits + row * a.d.logits_stride);
    // If `need` segments have j + 1 keys at or above a key each, and need (j + 1) >=
    // top, then nothing below it counts.  With need about half of the segments,
    // few more than `top` keys are left to order (32 segments' best 32: 6.0 us, all of
    // them ordered 18 us; no gain for 128 keys or fewer).
    __shared__ uint64_t ends[kMostSegments], least;
    uint32_t j = 0;
    while (j + 1 < top && (top + j) / (j + 1) > (segments + 1) / 2)
        ++j;
    const uint32_t need = (top + j) / (j + 1);
    const bool many = n_keys > 128;
    for (uint32_t i = threadIdx.x; i < segments && many; i += 256)
        ends[i] = keys[i * top + j];
    if (threadIdx.x == 0)
        least = 0;
    Best best;
    best.begin(list, sorted, &count, (int)top);
    if (many) {
        for (uint32_t i = threadIdx.x; i < segments; i += 256) {
            uint32_t above = 0;
#pragma unroll 8
            for (uint32_t k = 0; k < segments; ++k)
                above += ends[k] > ends[i];
            if (above + 1 == need)
                least = ends[i];
        }
        __syncthreads();
    }
    for (uint32_t base = 0; base < n_keys; base += 256) {
        const uint32_t q = base + threadIdx.x;
        const uint64_t key = q < n_keys ? keys[q] : 0;
        best.offer(key, key >= least);
        const uint32_t n = best.offered();
        if (n > kList - 256)
            best.order(n);
    }
    if (top > 0)
        best.order(best.offered());
    Part p{{kLowest, 0.0f, 0.0f}, 0};
    for (uint32_t i = threadIdx.x; i < segments; i += 256) {
        p.s.join(in[i].s);
        p.before += in[i].before;
    }
    p = over_workgroup(p, parts);
    put_scores(a, row, p, tk, sorted, best.kept);
}

// Rows of up to 512 K elements, a wave each, all in registers: no barrier, and
// the wave does no more than the row needs.  (In the kernel above three of four
// waves would have nothing, and no bound for the best.)  The bound is the value
// that `top` lanes reach with their largest; what reaches it, a few more than
// `top`, goes to LDS and is ordered.  Where that is more than kShortList (equal
// entries, more of `top` than lanes have entries), the last of the best is found
// bit by bit.  20000 x 1000 in bf16, 20 alternatives:
// 30 us (341 above, 23 with no alternatives); 4096 x 2048: 19 us, where 2049 take 30.
constexpr uint32_t kShortMost = 2048;
constexpr uint32_t kShortList = 128;

template <class T, int K> __global__ __launch_bounds__(256) void scores_short_kernel(ScoresArgs a)
{
    using raw = typename T::raw;
    __shared__ uint64_t lists[4][kShortList];
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t row = (int64_t)blockIdx.x * 4 + wave;
    if (row >= a.d.rows)
        return;
    const uint32_t V = (uint32_t)a.d.vocab;
    const raw *x = (const raw *)a.logits + row * a.d.logits_stride;
    // Pack 64 k + lane; the last one is loaded from an earlier start.
    Pack<T, 8> pack[K];
    uint32_t index[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t at = 8 * (64 * k + lane);
        index[k] = V < 8 ? at : at < V - 8 ? at : V - 8;
        if (V >= 8) {
            pack[k] = load_pack<T, 8>(x + index[k]);
        } else {
#pragma unroll
            for (uint32_t v = 0; v < 8; ++v)
                pack[k].v[v] = x[v < V ? v : V - 1];
        }
    }
    const Token tk = token_of<T>(a, row, x);
    const uint32_t mine = tk.known ? value_key(tk.value) : 0xFFFFFFFFu;
    const uint32_t id = tk.known ? (uint32_t)tk.id : 0;

    // keys, 0 where there is no entry
    uint32_t key[K][8], most = 0;
    float m = kLowest;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t at = 8 * (64 * k + lane);
#pragma unroll
        for (uint32_t v = 0; v < 8; ++v) {
            const bool real = index[k] + v >= at && index[k] + v < V;
            const float f = T::load(pack[k].v[v]);
            if (!real)
                pack[k].v[v] = T::store(-__builtin_inff());
            key[k][v] = real ? value_key(f) : 0;
            most = key[k][v] > most ? key[k][v] : most;
            m = __builtin_fmaxf(m, real ? f : m);
        }
    }
    Part p{{value_of(wave_max(value_key(m))), 0.0f, 0.0f}, 0};
    uint32_t before = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (uint32_t v = 0; v < 8; ++v) {
            const float d = T::load(pack[k].v[v]) - p.s.m;
            const float e = __builtin_amdgcn_exp2f(d * kLog2e);
            p.s.sum += e;
            p.s.cross = __builtin_fmaf(e, __builtin_fmaxf(d, kFar), p.s.cross);
            // (no key but 0 is below 1: equal entries of lower index come first)
            before += __popcll(__ballot(key[k][v] > mine - (index[k] + v < id)));
        }
    p.s.sum = wave_sum(p.s.sum);
    p.s.cross = wave_sum(p.s.cross);
    const float lse = __builtin_amdgcn_logf(p.s.sum) * kLn2;
    if (lane == 0) {
        if (a.logprob)
            a.logprob[row] = tk.known ? (tk.value - p.s.m) - lse : __uint_as_float(0x7FC00000u);
        if (a.entropy)
            a.entropy[row] = lse - p.s.cross / p.s.sum;
        if (a.rank)
            a.rank[row] = tk.known ? (int32_t)before : -1;
    }
    const uint32_t top = (uint32_t)a.d.top;
    if (top == 0)
        return;

    auto reach = [&](uint32_t t) {              // how many entries do
        uint32_t n = 0;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < 8; ++v)
                n += __popcll(__ballot(key[k][v] >= t));
        return n;
    };
    uint32_t t = 0, limit = ~0u;                // entries above t, or t at a lower index than limit
    for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit /= 2)
        if (__popcll(__ballot(most >= (t | bit))) >= (int)top)
            t |= bit;
    t = t > 0 ? t : 1;
    uint32_t n = reach(t);
    if (n > kShortList) {
        t = 0;
        for (uint32_t bit = 1u << 31; bit > 0; bit /= 2)
            if (reach(t | bit) >= top)
                t |= bit;
        // (nothing lies above a NaN, and more than kShortList entries are there, so that t > 0)
        const uint32_t wanted = t == ~0u ? top : top - reach(t + 1);
        limit = 0;                              // the largest below which there are fewer than wanted
        for (uint32_t bit = kShortMost / 2; bit > 0; bit /= 2) {
            uint32_t below = 0;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (uint32_t v = 0; v < 8; ++v)
                    below += __popcll(__ballot(key[k][v] == t && index[k] + v < (limit | bit)));
            if (below < wanted)
                limit |= bit;
        }
        ++limit;
        n = top;
    }
    uint64_t *list = lists[wave];
    uint32_t at = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (uint32_t v = 0; v < 8; ++v) {
            const uint32_t i = index[k] + v;
            const bool on = key[k][v] > t || (key[k][v] == t && i < limit);
            const uint64_t all = __ballot(on);
            if (on)
                list[at + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0))] =
                    ((uint64_t)key[k][v] << 32) | (0xFFFFFFFFu - i);
            at += __popcll(all);
        }
    // (a wave's accesses to LDS are in order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (uint32_t i = lane; i < n; i += 64) {
        const uint64_t mine = list[i];
        uint32_t place = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < n; ++j)
            place += list[j] > mine;
        if (place < top) {
            if (a.top_logprobs)
                a.top_logprobs[row * top + place] = (key_value(mine) - p.s.m) - lse;
            if (a.top_ids)
                a.top_ids[row * top + place] = (int32_t)key_index(mine);
        }
    }
    if (lane >= n && lane < top) {
        if (a.top_logprobs)
            a.top_logprobs[row * top + lane] = -__builtin_inff();
        if (a.top_ids)
            a.top_ids[row * top + lane] = -1;
    }
}

// Segments of a row: as many as bring about kMostSegments workgroups, of 8192
// elements or more each, if they save a workgroup more elements than a second
// launch takes (64 rows of 24000 in three 13.4 us, in one 11.0 us; 130 rows of
// 131072 in three 24.1 us, in one 26.1 us; 200 rows of 50000 in two 20.2 us, in one
// 16.0 us).
static uint32_t segments_of(const rnn_scores_desc &d, uint32_t &packs)
{
    const int64_t all = (d.vocab + 7) / 8;
    int64_t n = kMostSegments / d.rows;
    if (n > (all + 1023) / 1024)
        n = (all + 1023) / 1024;
    if (n < 1 || all / n * (n - 1) < 32768 / 8)
        n = 1;
    packs = (uint32_t)((all + n - 1) / n);
    return (uint32_t)((all + packs - 1) / packs);
}

size_t scores_workspace(const rnn_scores_desc &d)
{
    uint32_t packs;
    const uint32_t segments = segments_of(d, packs);
    return segments > 1 ? (size_t)d.rows * segments * (sizeof(Part) + 8 * (size_t)d.top) : 0;
}

template <class T> static int scores_go(const ScoresArgs &a, hipStream_t s)
{
    if (a.d.vocab <= kShortMost) {
        if (!launchable((uint64_t)(a.d.rows + 3) / 4, 256))
            return (int)hipErrorInvalidConfiguration;
        const dim3 grid((uint32_t)((a.d.rows + 3) / 4)), block(256);
        if (a.d.vocab <= 512)
            scores_short_kernel<T, 1><<<grid, block, 0, s>>>(a);
        else if (a.d.vocab <= 1024)
            scores_short_kernel<T, 2><<<grid, block, 0, s>>>(a);
        else
            scores_short_kernel<T, 4><<<grid, block, 0, s>>>(a);
        return (int)hipGetLastError();
    }
    uint32_t packs;
    const uint32_t segments = segments_of(a.d, packs);
    if (!launchable((uint64_t)a.d.rows * segments, 256))
        return (int)hipErrorInvalidConfiguration;
    scores_kernel<T><<<dim3((uint32_t)a.d.rows * segments), dim3(256), 0, s>>>(a, segments, packs);
    const int rc = (int)hipGetLastError();
    if (rc || segments == 1)
        return rc;
    scores_join_kernel<T><<<dim3((uint32_t)a.d.rows), dim3(256), 0, s>>>(a, segments);
    return (int)hipGetLastError();
}

int launch_scores(const ScoresArgs &a, hipStream_t s)
{
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: return scores_go<F32>(a, s);
    case RNN_DTYPE_BF16: return scores_go<BF16>(a, s);
    default: return scores_go<F16>(a, s);
    }
}

}  // namespace rnnamd
