// lm_run.cpp -- entry points of the language-model operators: every check
// before anything is enqueued, then the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <new>
#include <string>

#include "common.h"
#include "lm_common.h"

using namespace rnnamd;

namespace {

// What a check throws; nothing of it leaves the C entry points.
struct Fault {
    rnn_status status;
    std::string text;
};

[[noreturn]] void invalid(const std::string &text) { throw Fault{RNN_ERR_INVALID_INPUT, text}; }
[[noreturn]] void unsupported(const std::string &text) { throw Fault{RNN_ERR_UNSUPPORTED, text}; }

template <class F> rnn_status entry(const char *name, F &&body) noexcept
{
    try {
        set_error("");
        try {
            body();
            return RNN_OK;
        } catch (const Fault &f) {
            set_error(std::string(name) + ": " + f.text);
            return f.status;
        }
    } catch (...) {
        return RNN_ERR_OUT_OF_MEMORY;
    }
}

void launched(int rc)
{
    if (rc == (int)hipErrorInvalidConfiguration)
        unsupported("more work than one launch takes");
    if (rc)
        throw Fault{RNN_ERR_DEVICE, hipGetErrorString((hipError_t)rc)};
}

int64_t elem_size(int32_t dtype) { return dtype == RNN_DTYPE_F32 ? 4 : 2; }

void float_type(const char *name, int32_t dtype)
{
    if (dtype != RNN_DTYPE_F32 && dtype != RNN_DTYPE_BF16 && dtype != RNN_DTYPE_F16)
        invalid(std::string(name) + " must be RNN_DTYPE_F32, BF16 or F16");
}

void size_of(const char *name, int64_t v, int64_t lo = 0)
{
    if (v < lo || v > (int64_t)1 << 40)
        invalid(std::string(name) + " out of range: " + std::to_string(v));
}

void pointer(const char *name, const void *p, int64_t align, bool required = true)
{
    if (!p) {
        if (required)
            invalid(std::string(name) + " is required");
        return;
    }
    if ((uintptr_t)p % (uintptr_t)align)
        invalid(std::string(name) + " must be " + std::to_string(align) + "-byte aligned");
}

void workspace_of(const void *ws, size_t have, size_t need)
{
    if (need == 0)
        return;
    if (!ws || have < need)
        invalid("workspace missing or too small: " + std::to_string(need) + " bytes needed");
    if ((uintptr_t)ws % 256)
        invalid("workspace must be 256-byte aligned");
}

// Strides of a [n0, n1, inner] tensor: not negative, the extent countable; an
// output's elements must all be distinct.
void strides(const char *name, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner,
             bool output = false)
{
    if (n0 == 0 || n1 == 0 || inner == 0)
        return;
    const int64_t most = (int64_t)1 << 48;
    __int128 last = inner;
    if (n0 > 1)
        last += (__int128)(n0 - 1) * s0;
    if (n1 > 1)
        last += (__int128)(n1 - 1) * s1;
    if ((n0 > 1 && s0 < 0) || (n1 > 1 && s1 < 0) || last > most)
        invalid(std::string(name) + ": stride out of range");
    if (!output)
        return;
    const bool swap = n0 > 1 && n1 > 1 && s0 < s1;
    const int64_t in_n = swap ? n0 : n1, in_s = swap ? s0 : s1;
    const int64_t out_n = swap ? n1 : n0, out_s = swap ? s1 : s0;
    const int64_t span = in_n > 1 ? (in_n - 1) * in_s + inner : inner;
    if ((in_n > 1 && in_s < inner) || (out_n > 1 && out_s < span))
        invalid(std::string(name) + ": strides make its elements overlap");
}

void not_on(const char *out, const void *p, const char *in, const void *q)
{
    if (p && p == q)
        invalid(std::string(out) + " must not be " + in);
}

void check_scan(const rnn_scan_desc *d)
{
    if (!d)
        invalid("desc is required");
    size_of("batch", d->batch);
    size_of("steps", d->steps);
    size_of("dim", d->dim);
    if (d->states < 1 || d->states > RNN_SCAN_MAX_STATES)
        invalid("states must be 1 to " + std::to_string(RNN_SCAN_MAX_STATES));
    if (d->groups < 1 || d->dim % d->groups)
        invalid("groups must divide dim");
    float_type("dtype", d->dtype);
    if ((__int128)d->batch * d->steps > ((__int128)1 << 48) ||
        (__int128)d->batch * d->dim * d->states > ((__int128)1 << 48))
        invalid("sizes out of range");
    if (d->dim > 0x7fffffff || d->steps > 0x7fffffff)
        unsupported("more than 2^31 - 1 channels or steps");
}

void check_quant(const rnn_quant_desc *d)
{
    if (!d)
        invalid("desc is required");
    size_of("rows", d->rows);
    size_of("cols", d->cols);
    size_of("outs", d->outs);
    float_type("y_dtype", d->y_dtype);
    if (d->x_dtype != RNN_DTYPE_I8)
        float_type("x_dtype", d->x_dtype);
    if (d->cols > RNN_QUANT_MAX_COLS)
        unsupported("cols above " + std::to_string(RNN_QUANT_MAX_COLS) +
                    ": a 32-bit sum could overflow");
    if (d->rows >= ((int64_t)1 << 31) - 65536 || d->outs >= ((int64_t)1 << 31) - 65536)
        unsupported("2^31 - 2^16 rows or outs or more");
    strides("x", d->rows, d->x_stride, 1, 0, d->cols);
    strides("y", d->rows, d->y_stride, 1, 0, d->outs, true);
    if (d->outs > 0 && (d->w_stride < d->cols || d->w_stride % 16))
        invalid("w_stride must be a multiple of 16 and at least cols");
    strides("w", d->outs, d->w_stride, 1, 0, d->cols);
    if (d->x_dtype == RNN_DTYPE_I8 && d->rows > 0 && (d->x_stride < d->cols || d->x_stride % 16))
        invalid("x_stride of 8-bit rows must be a multiple of 16 and at least cols");
}

void check_scores(const rnn_scores_desc *d)
{
    if (!d)
        invalid("desc is required");
    size_of("rows", d->rows);
    size_of("vocab", d->vocab, 1);
    float_type("dtype", d->dtype);
    if (d->token_bytes != 4 && d->token_bytes != 8)
        invalid("token_bytes must be 4 or 8");
    if (d->top < 0 || d->top > RNN_SCORES_MAX_TOP)
        invalid("top must be 0 to " + std::to_string(RNN_SCORES_MAX_TOP));
    strides("logits", d->rows, d->logits_stride, 1, 0, d->vocab);
    if (d->rows > 0x7fffffff)
        unsupported("2^31 rows or more");
    if (d->vocab >= ((int64_t)1 << 31) - 65536)
        unsupported("vocab of 2^31 - 2^16 or more");
}

}  // namespace

extern "C" rnn_status rnn_conv_run(const rnn_conv_desc *d, void *hip_stream, const void *x,
                                   const float *weight, const float *bias, const void *state_in,
                                   const int32_t *lens, void *y, void *state_out)
{
    return entry("rnn_conv_run", [&] {
        if (!d)
            invalid("desc is required");
        size_of("batch", d->batch);
        size_of("steps", d->steps);
        size_of("dim", d->dim);
        if (d->taps < 1 || d->taps > RNN_CONV_MAX_TAPS)
            invalid("taps must be 1 to " + std::to_string(RNN_CONV_MAX_TAPS));
        float_type("dtype", d->dtype);
        strides("x", d->batch, d->x_batch_stride, d->steps, d->x_step_stride, d->dim);
        strides("y", d->batch, d->y_batch_stride, d->steps, d->y_step_stride, d->dim, true);
        const int64_t size = elem_size(d->dtype);
        const bool any = d->batch > 0 && d->dim > 0, some = any && d->steps > 0;
        pointer("x", x, size, some);
        pointer("weight", weight, 4, some);
        pointer("bias", bias, 4, false);
        pointer("state_in", state_in, size, false);
        pointer("sequence_lens", lens, 4, false);
        pointer("y", y, size, some);
        pointer("state_out", state_out, size, false);
        not_on("y", y, "x", x);
        not_on("y", y, "state_in", state_in);
        not_on("y", y, "state_out", state_out);
        not_on("state_out", state_out, "x", x);
        if (!any || (d->steps == 0 && (d->taps == 1 || !state_out)))
            return;
        launched(launch_conv(ConvArgs{*d, x, state_in, weight, bias, lens, y, state_out},
                             (hipStream_t)hip_stream));
    });
}

extern "C" rnn_status rnn_scan_workspace_size(const rnn_scan_desc *d, size_t *bytes)
{
    return entry("rnn_scan_workspace_size", [&] {
        check_scan(d);
        if (!bytes)
            invalid("bytes is required");
        *bytes = d->batch && d->dim ? scan_workspace(*d) : 0;
    });
}

extern "C" rnn_status rnn_scan_run(const rnn_scan_desc *d, void *hip_stream, void *workspace,
                                   size_t workspace_bytes, const void *x, const void *dt,
                                   const float *A, const void *B, const void *C, const float *D,
                                   const void *z, const float *dt_bias, const float *state_in,
                                   const int32_t *lens, void *y, float *state_out)
{
    return entry("rnn_scan_run", [&] {
        check_scan(d);
        strides("x", d->batch, d->x_batch_stride, d->steps, d->x_step_stride, d->dim);
        strides("dt", d->batch, d->dt_batch_stride, d->steps, d->dt_step_stride, d->dim);
        if (z)
            strides("z", d->batch, d->z_batch_stride, d->steps, d->z_step_stride, d->dim);
        strides("y", d->batch, d->y_batch_stride, d->steps, d->y_step_stride, d->dim, true);
        if (d->groups > 1) {
            strides("B", 1, 0, d->groups, d->B_group_stride, d->states);
            strides("C", 1, 0, d->groups, d->C_group_stride, d->states);
        }
        strides("B", d->batch, d->B_batch_stride, d->steps, d->B_step_stride, d->states);
        strides("C", d->batch, d->C_batch_stride, d->steps, d->C_step_stride, d->states);
        const int64_t size = elem_size(d->dtype);
        const bool any = d->batch > 0 && d->dim > 0, some = any && d->steps > 0;
        pointer("x", x, size, some);
        pointer("dt", dt, size, some);
        pointer("A", A, 4, some);
        pointer("B", B, size, some);
        pointer("C", C, size, some);
        pointer("D", D, 4, false);
        pointer("z", z, size, false);
        pointer("dt_bias", dt_bias, 4, false);
        pointer("state_in", state_in, 4, false);
        pointer("sequence_lens", lens, 4, false);
        pointer("y", y, size, some);
        pointer("state_out", state_out, 4, false);
        not_on("y", y, "x", x);
        not_on("y", y, "dt", dt);
        not_on("y", y, "z", z);
        not_on("y", y, "B", B);
        not_on("y", y, "C", C);
        not_on("y", y, "state_in", state_in);
        not_on("y", y, "state_out", state_out);
        if (!any || (d->steps == 0 && !state_out))
            return;
        workspace_of(workspace, workspace_bytes, scan_workspace(*d));
        launched(launch_scan(ScanArgs{*d, x, dt, B, C, z, A, D, dt_bias, state_in, lens, y,
                                      workspace, state_out},
                             (hipStream_t)hip_stream));
    });
}

extern "C" rnn_status rnn_quantize_rows(void *hip_stream, int64_t rows, int64_t cols,
                                        int32_t dtype, const void *x, int64_t x_stride, int8_t *q,
                                        int64_t q_stride, float *scale)
{
    return entry("rnn_quantize_rows", [&] {
        size_of("rows", rows);
        size_of("cols", cols);
        float_type("dtype", dtype);
        strides("x", rows, x_stride, 1, 0, cols);
        if (q_stride < cols || q_stride % 16)
            invalid("q_stride must be a multiple of 16 and at least cols");
        strides("q", rows, q_stride, 1, 0, q_stride, true);
        if (rows > 0x7fffffff)
            unsupported("2^31 rows or more");
        if (q_stride > (int64_t)1 << 30)
            unsupported("rows of more than 2^30 columns");
        if (rows == 0)
            return;
        pointer("x", x, elem_size(dtype), cols > 0);
        pointer("q", q, 16, q_stride > 0);
        pointer("scale", scale, 4);
        not_on("q", q, "x", x);
        launched(launch_quantize(QuantizeArgs{rows, cols, x_stride, q_stride, dtype, x, q, scale},
                                 (hipStream_t)hip_stream));
    });
}

extern "C" rnn_status rnn_quant_workspace_size(const rnn_quant_desc *d, size_t *bytes)
{
    return entry("rnn_quant_workspace_size", [&] {
        check_quant(d);
        if (!bytes)
            invalid("bytes is required");
        *bytes = d->rows && d->outs ? project_workspace(*d) : 0;
    });
}

extern "C" rnn_status rnn_quant_project(const rnn_quant_desc *d, void *hip_stream, void *workspace,
                                        size_t workspace_bytes, const void *x,
                                        const float *x_scale, const int8_t *w,
                                        const float *w_scale, const float *bias, void *y)
{
    return entry("rnn_quant_project", [&] {
        check_quant(d);
        if (d->rows == 0 || d->outs == 0)
            return;
        const bool eight = d->x_dtype == RNN_DTYPE_I8;
        pointer("x", x, eight ? 16 : elem_size(d->x_dtype), d->cols > 0);
        pointer("x_scale", x_scale, 4, eight);
        if (!eight && x_scale)
            invalid("x_scale must be NULL unless x is 8-bit");
        pointer("w", w, 16, d->cols > 0);
        pointer("w_scale", w_scale, 4);
        pointer("bias", bias, 4, false);
        pointer("y", y, elem_size(d->y_dtype));
        not_on("y", y, "x", x);
        workspace_of(workspace, workspace_bytes, project_workspace(*d));
        launched(launch_project(ProjectArgs{*d, x, x_scale, w_scale, bias, w, y, workspace},
                                (hipStream_t)hip_stream));
    });
}

extern "C" rnn_status rnn_scores_workspace_size(const rnn_scores_desc *d, size_t *bytes)
{
    return entry("rnn_scores_workspace_size", [&] {
        check_scores(d);
        if (!bytes)
            invalid("bytes is required");
        *bytes = d->rows ? scores_workspace(*d) : 0;
    });
}

extern "C" rnn_status rnn_token_scores(const rnn_scores_desc *d, void *hip_stream, void *workspace,
                                       size_t workspace_bytes, const void *logits,
                                       const void *tokens, float *logprob, float *entropy,
                                       int32_t *rank, float *top_logprobs, int32_t *top_ids)
{
    return entry("rnn_token_scores", [&] {
        check_scores(d);
        if (d->rows == 0)
            return;
        pointer("logits", logits, elem_size(d->dtype));
        pointer("tokens", tokens, d->token_bytes, logprob || rank);
        pointer("logprob", logprob, 4, false);
        pointer("entropy", entropy, 4, false);
        pointer("rank", rank, 4, false);
        pointer("top_logprobs", top_logprobs, 4, false);
        pointer("top_ids", top_ids, 4, false);
        workspace_of(workspace, workspace_bytes, scores_workspace(*d));
        launched(launch_scores(ScoresArgs{*d, logits, tokens, logprob, entropy, top_logprobs, rank,
                                          top_ids, workspace},
                               (hipStream_t)hip_stream));
    });
}
