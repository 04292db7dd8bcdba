// lm_beam.hip -- one step of beam search: the best continuations over the beams
// of each request and the vocabulary.
//
//   value(i, t) = scores[i] + x[i, t] - log sum_u exp(x[i, u])
//
// Bound by HBM: the logits are read once.  Within a beam the order is that of the
// logits themselves, so a workgroup keeps the sum of its segment of a beam and the
// first `keep` of its entries (from the maxima of eight parts of each thread's
// entries comes a bound that at least `keep` entries reach, and only parts that
// reach it are read again, from the caches).  A second launch sums the segments,
// and orders what they kept by the candidates' values, in float64: values of
// unlike beams lie next to each other, and a normaliser off by a rounding of
// float32 would decide between them.  Sums are taken in the order of the entries,
// whatever a row's alignment, so that equal beams have equal values and their
// candidates the order of the beams.
//
// 32 requests of 8 beams over 131072 entries in bf16 (67 MB, 13 us): 17.8 us, of which 7
// are the sums' own instructions (the vector unit is busy 40% of the cycles), and 5.2 us for
// the join, a chain of a read, the sums and the ranks.  One request of 4 beams over 100001
// in f32: 7.2 and 6.9 us, a few trips to memory each and the launch.
#include <type_traits>

#include "lm_order.h"

namespace rnnamd {

constexpr float kLow = -3.402823466e38f;

struct Total {              // sum exp(x - m)
    double sum;
    float m;
    __device__ __forceinline__ void rebase(float to)
    {
        sum *= exp((double)m - (double)to);
        m = to;
    }
};

// A beam whose entries count: not finished, and with a finite score.
__device__ __forceinline__ bool beam_runs(const BeamArgs &a, int64_t row)
{
    const float s = a.scores[row];
    return s - s == 0.0f && !(a.finished && a.finished[row]);
}

// One segment of a beam's row: packs [first, last) of 8 entries.  A thread takes
// every 256th pack, U at a time: the loads of a batch are in flight while the one
// before is summed.
template <class T> __global__ __launch_bounds__(256) void beam_rows_kernel(BeamArgs a, uint32_t segments,
                                                                         uint32_t segment_packs)
{
    using raw = typename T::raw;
    constexpr uint32_t PARTS = 8, U = sizeof(raw) == 2 ? 4 : 2, BATCH = 256 * U;
    constexpr int WORDS = 8 * sizeof(raw) / 4;
    __shared__ uint64_t list[kList], sorted[RNN_SCORES_MAX_TOP];
    __shared__ float most[PARTS][256];
    __shared__ uint32_t count, bounds[4];
    __shared__ uint16_t items[256];
    __shared__ uint8_t finite[4];
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int64_t row = blockIdx.x / segments;
    const uint32_t segment = blockIdx.x % segments;
    if (!beam_runs(a, row))
        return;
    const raw *x = (const raw *)a.logits + row / a.d.beams * a.d.logits_batch_stride +
                   row % a.d.beams * a.d.logits_beam_stride;
    const uint32_t V = (uint32_t)a.d.vocab, all = (V + 7) / 8;
    const uint32_t first = segment * segment_packs;
    const uint32_t last = first + segment_packs < all ? first + segment_packs : all;
    const uint32_t whole = last < V / 8 ? last : V / 8;      // packs of all 8 entries end here
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

    Total p{0.0, kLow};
    float top_of_part = -__builtin_inff(), top_of_all = top_of_part;
    auto one = [&](const float (&f)[8]) {
        const float pm = __builtin_fmaxf(
            __builtin_fmaxf(__builtin_fmaxf(f[0], f[1]), __builtin_fmaxf(f[2], f[3])),
            __builtin_fmaxf(__builtin_fmaxf(f[4], f[5]), __builtin_fmaxf(f[6], f[7])));
        top_of_part = __builtin_fmaxf(top_of_part, pm);
        if (__builtin_expect(__ballot(pm > p.m) != 0, 0)) {     // a few times a row
            const float to = value_of(wave_max(value_key(pm)));
            p.rebase(to > p.m ? to : p.m);
        }
        float e[8];
#pragma unroll
        for (int v = 0; v < 8; ++v)
            e[v] = __builtin_amdgcn_exp2f((f[v] - p.m) * kLog2e);
        p.sum += (double)(((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
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
            one(f);
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
    // the last entries, fewer than a pack, one a thread
    const uint32_t rest = last * 8 > V ? V - whole * 8 : 0;
    const float f_rest = tid < rest ? T::load(x[whole * 8 + tid]) : -__builtin_inff();
    if (wave == 0 && rest > 0) {
        float f[8];
#pragma unroll
        for (int v = 1; v < 8; ++v)
            f[v] = -__builtin_inff();
        f[0] = f_rest;
        one(f);
        top_of_all = __builtin_fmaxf(top_of_all, f_rest);
    }
    // a wave's lanes have the same m
    p.sum = sums_up_to(p.sum);
    const int top = a.d.keep;
    uint64_t *keys = (uint64_t *)a.workspace + (int64_t)blockIdx.x * top;
    Total *out = (Total *)((uint64_t *)a.workspace + (int64_t)gridDim.x * top) + 4 * (int64_t)blockIdx.x;
    if (lane == 63) {
        out[wave] = p;
        finite[wave] = p.sum < (double)__builtin_inff();
    }
    Best best;
    best.begin(list, sorted, &count, top);
    // The bound, to 16 bits: the largest t that enough lanes of each wave reach.
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
    // NaN or infinite entries: the beam has no distribution, its entries do not count
    if (!(finite[0] && finite[1] && finite[2] && finite[3]))
        return;
    // (cut to 16 bits, -inf lies below every number's key)
    const float edge = t < value_key(kLow) ? -__builtin_inff() : value_of(t);
    if (batches > 0)
        for (uint32_t s = 0; s < PARTS; ++s)
            if (most[s][tid] >= edge) {
                const uint32_t at = atomicAdd(&count, 1u);
                if (at < 256)
                    items[at] = (uint16_t)(s * 256 + tid);
            }
    uint32_t n = best.offered();
    best.forget();
    const bool few = n <= 256;
    const uint32_t item_packs = part_batches * U;
    const uint32_t packs = few ? n * item_packs : last - first;
    if (few)
        best.offer(order_key(f_rest, whole * 8 + tid), tid < rest && f_rest >= edge);
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
        uint64_t some[8];
        uint32_t want = 0;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            const float f = T::load(pk.v[v]);
            some[v] = order_key(f, 8 * i + v);
            want |= (uint32_t)(on && 8 * i + v < V && f >= edge) << v;
        }
        best.offer(some, want);
        n = best.offered();
        if (n > kList) {            // too many at once: an eighth of them at a time
            best.forget();
#pragma unroll 1
            for (int v = 0; v < 8; ++v) {
                const float f = T::load(pk.v[0]);
                best.offer(order_key(f, 8 * i + v), on && 8 * i + v < V && f >= edge);
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
    if (tid < (uint32_t)top)
        keys[tid] = tid < best.kept ? sorted[tid] : 0;
}

// A candidate: its value as a number that orders as it does (0: none), and its
// place i vocab + t.  (float64 has no -0 here: a sum of a number and +0 or -0.)
struct Candidate {
    uint64_t value, place;
    __device__ __forceinline__ bool before(const Candidate &o) const
    {
        return value != o.value ? value > o.value : place < o.place;
    }
};
__device__ __forceinline__ uint64_t double_key(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    return (u >> 63) ? ~u : (u | 1ull << 63);
}
__device__ __forceinline__ double key_double(uint64_t u)
{
    return __builtin_bit_cast(double, (u >> 63) ? u ^ 1ull << 63 : ~u);
}

constexpr uint32_t kMostLists = 512;

// The beams of a request together; `lists`: segments of all beams, up to
// kMostLists, each with its first `keep` entries in order.
__global__ __launch_bounds__(256) void beam_join_kernel(BeamArgs a, uint32_t segments)
{
    constexpr uint32_t LIST = 512;
    __shared__ double base[RNN_BEAM_MAX];           // what a beam's candidates have beside x
    __shared__ uint8_t kind[RNN_BEAM_MAX];          // 0: dead, 1: runs, 2: finished
    __shared__ uint64_t ends[kMostLists], least;
    __shared__ Total sums[4 * kMostLists];
    __shared__ float most[RNN_BEAM_MAX];
    __shared__ Candidate list[LIST], sorted[RNN_BEAM_MAX];
    __shared__ uint32_t count;
    const uint32_t tid = threadIdx.x, keep = (uint32_t)a.d.keep, beams = (uint32_t)a.d.beams;
    const uint32_t lists = beams * segments;
    const uint64_t V = (uint64_t)a.d.vocab, eos = (uint64_t)a.d.eos;
    const int64_t first_row = (int64_t)blockIdx.x * beams;
    const uint64_t *keys = (const uint64_t *)a.workspace + first_row * segments * keep;
    const Total *totals = (const Total *)((const uint64_t *)a.workspace +
                                          (int64_t)gridDim.x * beams * segments * keep) +
                          first_row * segments * 4;
    const uint32_t all = lists * keep;
    // If `need` lists have j + 1 candidates at or above a value each, and need (j + 1)
    // >= keep, then nothing below it counts.  With need about half of the lists, few
    // more than `keep` are left to order.
    uint32_t j = 0;
    while (j + 1 < keep && (keep + j) / (j + 1) > (lists + 1) / 2)
        ++j;
    const uint32_t need = (keep + j) / (j + 1);
    // (keys that come while the sums are joined: the first ones, and those of `ends`)
    constexpr uint32_t FIRST = 4;
    uint64_t my_key[FIRST], end_key[kMostLists / 256];
#pragma unroll
    for (uint32_t i = 0; i < FIRST; ++i)
        my_key[i] = keys[tid + 256 * i < all ? tid + 256 * i : 0];
#pragma unroll
    for (uint32_t i = 0; i < kMostLists / 256; ++i)
        end_key[i] = keys[tid + 256 * i < lists ? (tid + 256 * i) * keep + j : 0];
    if (tid == 0) {
        count = 0;
        least = 0;
    }
    // every wave's sum by itself, then the beams': exponentials are long in float64
    const uint32_t waves = 4 * segments, parts = beams * waves;
    for (uint32_t i = tid; i < parts; i += 256)
        sums[i] = beam_runs(a, first_row + i / waves) ? totals[i] : Total{0.0, kLow};
    if (tid < beams) {
        const int64_t row = first_row + tid;
        const float score = a.scores[row];
        base[tid] = score;
        kind[tid] = score - score == 0.0f ? a.finished && a.finished[row] ? 2 : 1 : 0;
    }
    __syncthreads();
    if (tid < beams) {
        float m[4] = {kLow, kLow, kLow, kLow};  // (waves is a multiple of 4)
#pragma unroll 4
        for (uint32_t s = 0; s < waves; s += 4)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                m[v] = __builtin_fmaxf(m[v], sums[tid * waves + s + v].m);
        most[tid] = __builtin_fmaxf(__builtin_fmaxf(m[0], m[1]), __builtin_fmaxf(m[2], m[3]));
    }
    __syncthreads();
    for (uint32_t i = tid; i < parts; i += 256) {
        Total o = sums[i];
        o.rebase(most[i / waves]);
        sums[i].sum = o.sum;
    }
    __syncthreads();
    if (tid < beams && kind[tid] == 1) {
        double sum[4] = {};
#pragma unroll 4
        for (uint32_t s = 0; s < waves; s += 4)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                sum[v] += sums[tid * waves + s + v].sum;
        const double c = base[tid] - ((double)most[tid] + log((sum[0] + sum[1]) + (sum[2] + sum[3])));
        base[tid] = c;
        kind[tid] = c - c == 0.0;
    }
    __syncthreads();
    // entry e of list l, whose key (of a beam that runs) is `key`
    auto candidate = [&](uint32_t l, uint32_t e, uint64_t key) {
        const uint32_t beam = l / segments;
        const uint64_t row = beam * V, none = double_key(-(double)__builtin_inff());
        if (kind[beam] == 1) {
            if (key == 0)
                return Candidate{0, ~0ull};
            return Candidate{double_key(base[beam] + (double)key_value(key)), row + key_index(key)};
        }
        if (l % segments)
            return Candidate{0, ~0ull};
        uint64_t token = e;
        if (kind[beam] == 2) {
            if (e == 0)
                return Candidate{double_key(base[beam]), row + eos};
            token = e - 1 < eos ? e - 1 : e;
        }
        return token < V ? Candidate{none, row + token} : Candidate{0, ~0ull};
    };
    if (all > 64) {
#pragma unroll
        for (uint32_t i = 0; i < kMostLists / 256; ++i)
            if (tid + 256 * i < lists)
                ends[tid + 256 * i] = candidate(tid + 256 * i, j, end_key[i]).value;
        __syncthreads();
        for (uint32_t i = tid; i < lists; i += 256) {
            uint32_t above = 0, equal = 0;
#pragma unroll 8
            for (uint32_t k = 0; k < lists; ++k) {
                above += ends[k] > ends[i];
                equal += ends[k] == ends[i];
            }
            if (above < need && need <= above + equal)
                least = ends[i];                    // (the same from all that write)
        }
        __syncthreads();
    }
    const uint64_t bound = least;
    uint32_t kept = 0;
    Candidate worst{0, ~0ull};                      // the last of `keep` kept ones
    auto order = [&]() {
        __syncthreads();
        const uint32_t n = count < LIST ? count : LIST;
        // a candidate's place is the number of those before it: four lanes, or one
        const uint32_t lanes = n <= 64 ? 4 : 1;
        for (uint32_t i = tid / lanes; i < n; i += 256) {
            const Candidate mine = list[i];
            uint32_t place = 0;
#pragma unroll 4
            for (uint32_t k = tid % lanes; k < n; k += lanes)
                place += list[k].before(mine);
            if (lanes == 4) {
                place += __shfl_xor(place, 1);
                place += __shfl_xor(place, 2);
            }
            if (place < keep)
                sorted[place] = mine;
        }
        __syncthreads();
        kept = n < keep ? n : keep;
        if (tid < kept)
            list[tid] = sorted[tid];
        if (tid == 0)
            count = kept;
        if (n >= keep)
            worst = sorted[keep - 1];
        __syncthreads();
    };
    auto offer = [&](uint32_t q, uint64_t key) {
        if (q < all) {
            const Candidate c = candidate(q / keep, q % keep, key);
            if (c.value != 0 && c.value >= bound && c.before(worst))
                list[atomicAdd(&count, 1u)] = c;
        }
        __syncthreads();
        const uint32_t n = count;
        __syncthreads();
        if (n > LIST - 256)
            order();
    };
#pragma unroll
    for (uint32_t i = 0; i < FIRST; ++i)
        if (256 * i < all)
            offer(tid + 256 * i, my_key[i]);
    for (uint32_t from = 256 * FIRST; from < all; from += 256)
        offer(from + tid, from + tid < all ? keys[from + tid] : 0);
    order();
    if (tid < keep) {
        const bool have = tid < kept;
        const Candidate c = have ? sorted[tid] : Candidate{0, 0};
        const int64_t at = (int64_t)blockIdx.x * keep + tid;
        a.out_scores[at] = have ? (float)key_double(c.value) : -__builtin_inff();
        a.out_tokens[at] = have ? (int32_t)(c.place % V) : -1;
        a.out_parents[at] = have ? (int32_t)(c.place / V) : -1;
    }
}

// Segments of a row: as many as bring about 512 workgroups, of 8192 entries or more
// each, and no more lists than the join orders well.  Both kernels' time, us: 512
// workgroups against 256 and 1024: 32 x 8 beams x 131072 bf16 24.4, 26.9, 26.8; 8 x 5 x
// 262144 18.5, 18.3, 23.4.  8192 entries against 4096 and 16384: 1 x 4 x 100001 f32 14.0,
// 15.8, 14.4; 1 x 16 x 32000 bf16 14.6, 18.6, 14.2; 128 x 4 x 8000 f16 13.5, 13.7, 14.9.
static uint32_t beam_segments(const rnn_beam_desc &d, uint32_t &packs)
{
    const int64_t all = (d.vocab + 7) / 8, rows = d.batch * d.beams;
    int64_t n = 512 / rows;
    if (n > (all + 1023) / 1024)
        n = (all + 1023) / 1024;
    if (n > kMostLists / d.beams)
        n = kMostLists / d.beams;
    if (n < 1)
        n = 1;
    packs = (uint32_t)((all + n - 1) / n);
    return (uint32_t)((all + packs - 1) / packs);
}

size_t beam_workspace(const rnn_beam_desc &d)
{
    uint32_t packs;
    return (size_t)d.batch * d.beams * beam_segments(d, packs) * (4 * sizeof(Total) + 8 * (size_t)d.keep);
}

template <class T> static int beam_go(const BeamArgs &a, hipStream_t s)
{
    uint32_t packs;
    const uint32_t segments = beam_segments(a.d, packs);
    const uint64_t blocks = (uint64_t)a.d.batch * a.d.beams * segments;
    if (!launchable(blocks, 256))
        return (int)hipErrorInvalidConfiguration;
    beam_rows_kernel<T><<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(a, segments, packs);
    const int rc = (int)hipGetLastError();
    if (rc)
        return rc;
    beam_join_kernel<<<dim3((uint32_t)a.d.batch), dim3(256), 0, s>>>(a, segments);
    return (int)hipGetLastError();
}

int launch_beam(const BeamArgs &a, hipStream_t s)
{
    switch (a.d.dtype) {
    case RNN_DTYPE_F32: return beam_go<F32>(a, s);
    case RNN_DTYPE_BF16: return beam_go<BF16>(a, s);
    default: return beam_go<F16>(a, s);
    }
}

}  // namespace rnnamd
