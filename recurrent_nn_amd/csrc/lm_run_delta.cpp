// lm_run_delta.cpp -- entry points of the delta-rule operators and of decoding
// with several beams: every check before anything is enqueued, then the
// launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "lm_checks.h"
#include "lm_common.h"

using namespace rnnamd;

namespace {

// Strides of [n0, n1, n2, inner], as strides() for three of them.
void strides3(const char *name, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2,
              int64_t inner, bool output = false)
{
    if (n0 == 0 || n1 == 0 || n2 == 0 || inner == 0)
        return;
    const int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2}, most = (int64_t)1 << 48;
    __int128 last = inner;
    for (int i = 0; i < 3; ++i) {
        if (n[i] > 1 && s[i] < 0)
            invalid(std::string(name) + ": stride out of range");
        if (n[i] > 1)
            last += (__int128)(n[i] - 1) * s[i];
    }
    if (last > most)
        invalid(std::string(name) + ": stride out of range");
    if (!output)
        return;
    // from the smallest stride on, each beyond what the ones before it span
    bool done[3] = {n0 == 1, n1 == 1, n2 == 1};
    int64_t span = inner;
    for (;;) {
        int at = -1;
        for (int i = 0; i < 3; ++i)
            if (!done[i] && (at < 0 || s[i] < s[at]))
                at = i;
        if (at < 0)
            return;
        if (s[at] < span)
            invalid(std::string(name) + ": strides make its elements overlap");
        span += (n[at] - 1) * s[at];
        done[at] = true;
    }
}

void check_delta(const rnn_delta_desc *d)
{
    if (!d)
        invalid("desc is required");
    size_of("batch", d->batch);
    size_of("steps", d->steps);
    size_of("heads", d->heads);
    size_of("value_dim", d->value_dim);
    if (d->key_heads < 1 || d->heads % d->key_heads)
        invalid("key_heads must divide heads");
    if (d->key_dim < 1 || d->key_dim > RNN_DELTA_MAX_KEY_DIM)
        invalid("key_dim must be 1 to " + std::to_string(RNN_DELTA_MAX_KEY_DIM));
    float_type("dtype", d->dtype);
    if (d->gate_dtype != RNN_DTYPE_F32 && d->gate_dtype != d->dtype)
        invalid("gate_dtype must be F32 or dtype");
    if (!std::isfinite(d->scale))
        invalid("scale must be finite");
    const __int128 most = (__int128)1 << 48;
    if ((__int128)d->batch * d->steps > most || (__int128)d->batch * d->heads > most ||
        (__int128)d->batch * d->heads * d->key_dim > most ||
        (__int128)d->batch * d->heads * d->key_dim * d->value_dim > most ||
        (__int128)d->batch * d->steps * d->heads > most)
        invalid("sizes out of range");
    if (d->steps > 0x7fffffff || d->heads > 0x7fffffff || d->value_dim > 0x7fffffff)
        unsupported("2^31 steps, heads or columns or more");
}

void check_beam(const rnn_beam_desc *d)
{
    if (!d)
        invalid("desc is required");
    size_of("batch", d->batch);
    size_of("vocab", d->vocab, 1);
    if (d->beams < 1 || d->beams > RNN_BEAM_MAX)
        invalid("beams must be 1 to " + std::to_string(RNN_BEAM_MAX));
    if (d->keep < 1 || d->keep > RNN_BEAM_MAX)
        invalid("keep must be 1 to " + std::to_string(RNN_BEAM_MAX));
    float_type("dtype", d->dtype);
    strides("logits", d->batch, d->logits_batch_stride, d->beams, d->logits_beam_stride, d->vocab);
    if (d->vocab >= ((int64_t)1 << 31) - 65536)
        unsupported("vocab of 2^31 - 2^16 or more");
}

// What a call reads or writes, from its first byte to behind its last.
struct Stretch {
    uintptr_t from, to;
    bool written;
};

// What is written lies on nothing else.
void apart(std::vector<Stretch> &all)
{
    std::sort(all.begin(), all.end(), [](const Stretch &x, const Stretch &y) { return x.from < y.from; });
    uintptr_t read = 0, written = 0;            // the ends so far
    for (const Stretch &s : all) {
        if (s.from < written || (s.written && s.from < read))
            invalid("an item's out overlaps another item or parents");
        uintptr_t &end = s.written ? written : read;
        end = std::max(end, s.to);
    }
}

}  // namespace

extern "C" rnn_status rnn_delta_workspace_size(const rnn_delta_desc *d, size_t *bytes)
{
    return entry("rnn_delta_workspace_size", [&] {
        check_delta(d);
        if (!bytes)
            invalid("bytes is required");
        *bytes = d->batch && d->heads && d->value_dim ? delta_workspace(*d) : 0;
    });
}

extern "C" rnn_status rnn_delta_run(const rnn_delta_desc *d, void *hip_stream, void *workspace,
                                    size_t workspace_bytes, const void *q, const void *k,
                                    const void *v, const void *beta, const void *g, const float *A,
                                    const float *dt_bias, const float *state_in,
                                    const int32_t *lens, void *o, float *state_out)
{
    return entry("rnn_delta_run", [&] {
        check_delta(d);
        strides3("q", d->batch, d->q_batch_stride, d->steps, d->q_step_stride, d->key_heads,
                 d->q_head_stride, d->key_dim);
        strides3("k", d->batch, d->k_batch_stride, d->steps, d->k_step_stride, d->key_heads,
                 d->k_head_stride, d->key_dim);
        strides3("v", d->batch, d->v_batch_stride, d->steps, d->v_step_stride, d->heads,
                 d->v_head_stride, d->value_dim);
        strides3("o", d->batch, d->o_batch_stride, d->steps, d->o_step_stride, d->heads,
                 d->o_head_stride, d->value_dim, true);
        strides("beta", d->batch, d->beta_batch_stride, d->steps, d->beta_step_stride, d->heads);
        if (g)
            strides("g", d->batch, d->g_batch_stride, d->steps, d->g_step_stride, d->heads);
        const int64_t size = elem_size(d->dtype), gate = elem_size(d->gate_dtype);
        const bool any = d->batch > 0 && d->heads > 0 && d->value_dim > 0, some = any && d->steps > 0;
        pointer("q", q, size, some);
        pointer("k", k, size, some);
        pointer("v", v, size, some);
        pointer("beta", beta, gate, some);
        pointer("g", g, gate, false);
        pointer("A", A, 4, false);
        pointer("dt_bias", dt_bias, 4, false);
        if (some && A && !g)
            invalid("A needs g");
        if (some && dt_bias && !A)
            invalid("dt_bias needs A");
        pointer("state_in", state_in, 4, false);
        pointer("sequence_lens", lens, 4, false);
        pointer("o", o, size, some);
        pointer("state_out", state_out, 4, false);
        not_on("o", o, "q", q);
        not_on("o", o, "k", k);
        not_on("o", o, "v", v);
        not_on("o", o, "beta", beta);
        not_on("o", o, "g", g);
        not_on("o", o, "state_in", state_in);
        not_on("o", o, "state_out", state_out);
        if (!any || (d->steps == 0 && !state_out))
            return;
        workspace_of(workspace, workspace_bytes, delta_workspace(*d));
        launched(launch_delta(DeltaArgs{*d, q, k, v, beta, g, A, dt_bias, state_in, lens, o, workspace,
                                        state_out},
                              (hipStream_t)hip_stream));
    });
}

extern "C" rnn_status rnn_gated_norm(const rnn_norm_desc *d, void *hip_stream, const void *x,
                                     const float *weight, const void *z, void *y)
{
    return entry("rnn_gated_norm", [&] {
        if (!d)
            invalid("desc is required");
        size_of("rows", d->rows);
        size_of("groups", d->groups);
        size_of("dim", d->dim);
        float_type("dtype", d->dtype);
        if (!(d->eps >= 0.0f) || !std::isfinite(d->eps))
            invalid("eps must be 0 or more and finite");
        strides("x", d->rows, d->x_row_stride, d->groups, d->x_group_stride, d->dim);
        if (z)
            strides("z", d->rows, d->z_row_stride, d->groups, d->z_group_stride, d->dim);
        strides("y", d->rows, d->y_row_stride, d->groups, d->y_group_stride, d->dim, true);
        strides("weight", d->groups, d->weight_group_stride, 1, 0, d->dim);
        if (d->gate_first && !z)
            invalid("gate_first needs z");
        if (d->dim >= (int64_t)1 << 30 || d->groups > 0x7fffffff)
            unsupported("a dim of 2^30 or more, or 2^31 groups or more");
        const bool some = d->rows > 0 && d->groups > 0 && d->dim > 0;
        const int64_t size = elem_size(d->dtype);
        pointer("x", x, size, some);
        pointer("weight", weight, 4, some);
        pointer("z", z, size, false);
        pointer("y", y, size, some);
        const auto in_place = [&](const char *name, const void *p, int64_t row, int64_t group) {
            if (p && p == y && ((d->rows > 1 && row != d->y_row_stride) ||
                                (d->groups > 1 && group != d->y_group_stride)))
                invalid(std::string("y on ") + name + " must have its strides");
        };
        in_place("x", x, d->x_row_stride, d->x_group_stride);
        in_place("z", z, d->z_row_stride, d->z_group_stride);
        if (!some)
            return;
        launched(launch_norm(NormArgs{*d, x, z, weight, y}, (hipStream_t)hip_stream));
    });
}

extern "C" rnn_status rnn_beam_workspace_size(const rnn_beam_desc *d, size_t *bytes)
{
    return entry("rnn_beam_workspace_size", [&] {
        check_beam(d);
        if (!bytes)
            invalid("bytes is required");
        *bytes = d->batch ? beam_workspace(*d) : 0;
    });
}

extern "C" rnn_status rnn_beam_select(const rnn_beam_desc *d, void *hip_stream, void *workspace,
                                      size_t workspace_bytes, const void *logits,
                                      const float *scores, const uint8_t *finished,
                                      float *out_scores, int32_t *out_tokens, int32_t *out_parents)
{
    return entry("rnn_beam_select", [&] {
        check_beam(d);
        if (finished && (d->eos < 0 || d->eos >= d->vocab))
            invalid("eos must be in [0, vocab)");
        const bool some = d->batch > 0;
        pointer("logits", logits, elem_size(d->dtype), some);
        pointer("scores", scores, 4, some);
        pointer("out_scores", out_scores, 4, some);
        pointer("out_tokens", out_tokens, 4, some);
        pointer("out_parents", out_parents, 4, some);
        not_on("out_scores", out_scores, "scores", scores);
        not_on("out_tokens", out_tokens, "out_parents", out_parents);
        if (!some)
            return;
        workspace_of(workspace, workspace_bytes, beam_workspace(*d));
        launched(launch_beam(BeamArgs{*d, logits, scores, finished, out_scores, out_tokens, out_parents,
                                      workspace},
                             (hipStream_t)hip_stream));
    });
}

extern "C" rnn_status rnn_reorder_states(void *hip_stream, int64_t batch, int64_t beams, int64_t keep,
                                         const int32_t *parents, const rnn_reorder_item *items,
                                         int64_t count)
{
    return entry("rnn_reorder_states", [&] {
        size_of("batch", batch);
        size_of("beams", beams, 1);
        size_of("keep", keep);
        size_of("count", count);
        if ((__int128)batch * beams > ((__int128)1 << 40) || (__int128)batch * keep > ((__int128)1 << 40))
            invalid("sizes out of range");
        const bool some = batch > 0 && keep > 0 && count > 0;
        pointer("parents", parents, 4, some);
        if (count > 0 && !items)
            invalid("items are required");
        std::vector<Stretch> all;
        all.reserve(2 * count + 1);
        all.push_back({(uintptr_t)parents, (uintptr_t)parents + (uintptr_t)(4 * batch * keep), false});
        for (int64_t i = 0; i < count; ++i) {
            const rnn_reorder_item &it = items[i];
            size_of("outer", it.outer);
            size_of("inner_bytes", it.inner_bytes);
            const __int128 most = (__int128)1 << 48, row = (__int128)it.outer * it.inner_bytes;
            if (row * batch * beams > most || row * batch * keep > most)
                invalid("sizes out of range");
            const int64_t from = (int64_t)(row * batch * beams), to = (int64_t)(row * batch * keep);
            if (to == 0)
                continue;
            pointer("in", it.in, 1);
            pointer("out", it.out, 1);
            if (it.in == it.out) {
                if (keep != beams)
                    invalid("in place needs keep = beams");
                if (beams > RNN_REORDER_MAX_BEAMS)
                    unsupported("in place with more than " + std::to_string(RNN_REORDER_MAX_BEAMS) +
                                " beams");
            } else if ((uintptr_t)it.in < (uintptr_t)it.out + (uintptr_t)to &&
                       (uintptr_t)it.out < (uintptr_t)it.in + (uintptr_t)from) {
                invalid("out overlaps in");
            }
            all.push_back({(uintptr_t)it.out, (uintptr_t)it.out + (uintptr_t)to, true});
            if (it.in != it.out)
                all.push_back({(uintptr_t)it.in, (uintptr_t)it.in + (uintptr_t)from, false});
        }
        apart(all);
        if (!some)
            return;
        ReorderArgs a{batch, beams, keep, parents, 0, {}, {}};
        // (everything is checked before the first launch)
        for (int pass = 0; pass < 2; ++pass) {
            a.count = 0;
            for (int64_t i = 0; i < count; ++i) {
                if (items[i].outer > 0 && items[i].inner_bytes > 0)
                    a.items[a.count++] = items[i];
                if (a.count == kReorderItems || (i == count - 1 && a.count > 0)) {
                    if (pass == 0)
                        launched(reorder_fits(a));
                    else
                        launched(launch_reorder(a, (hipStream_t)hip_stream));
                    a.count = 0;
                }
            }
        }
    });
}
