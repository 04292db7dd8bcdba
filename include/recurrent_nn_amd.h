/*
 * recurrent_nn_amd.h -- C-ABI of the MI355X (gfx950) implementation of the
 * ONNX recurrent operators RNN, GRU and LSTM.
 *
 * What is computed is defined on the onemodel page "Recurrent operators: RNN,
 * GRU, LSTM":
 *   - gate packing (LSTM i,o,f,c; GRU z,r,h; B = [W biases, R biases];
 *     P = [i, o, f] peepholes) ..................... section "Support"
 *   - XW = X . W^T over all steps, the per-step H . R^T, the gate arithmetic
 *     in its written order ........................ section "Computation"
 *   - activations, their parameters and cursors ... section "Activations"
 *   - sequence_lens, input_forget, layout 1, omitted inputs, zero-size,
 *     hidden_size .................................. section "Choices the
 *                                                     specification leaves open"
 *   - every NaN written as 0x7FC00000 ............. section "Exact mode"
 *   - fused multiply-add only inside the products . section "Fast mode"
 *   - scratch limit, Unsupported at plan time ..... section "Limits"
 * The input/output tables (shapes for layout 0 and 1, float32 T, int32
 * sequence_lens) are those of the WebGPU "ai.onnx.RNN" package README,
 * sections "Inputs", "Outputs", "Attributes", "Type constraints".
 *
 * This library runs the "fast mode" order: the two products (projection and
 * recurrent product) accumulate in the matrix cores' order with a fixed
 * tiling, so results are deterministic run to run; every other operation is
 * the written IEEE binary32 operation, unfused, in the written order.
 *
 * Conventions for every entry point
 *   - Tensors are dense row-major float32 in ONNX shapes for the attribute
 *     `layout` (layout 0: X [seq, batch, input], initial states and Y_h/Y_c
 *     [dirs, batch, hidden], Y [seq, dirs, batch, hidden]; layout 1: X
 *     [batch, seq, input], states [batch, dirs, hidden], Y [batch, seq, dirs,
 *     hidden]).  W is [dirs, G*hidden, input], R [dirs, G*hidden, hidden],
 *     B [dirs, 2*G*hidden], P [dirs, 3*hidden]; G = 1 (RNN), 3 (GRU), 4 (LSTM).
 *   - Every tensor pointer given to rnn_run is a DEVICE pointer on the current
 *     HIP device, except sequence_lens, which is a HOST int32 array (so that the
 *     range check is synchronous).  Device pointers must be 16-byte aligned.
 *   - The caller owns every tensor and the workspace; the plan owns host
 *     memory only.  rnn_run is stream-ordered and asynchronous: keep the
 *     tensors and the workspace alive until the stream has passed the work.
 *   - A plan with one workspace serves one stream at a time; concurrent runs
 *     need distinct workspaces.
 *   - Every check happens before anything is enqueued: a non-OK status leaves
 *     every output untouched.  rnn_last_error() then describes the failure.
 */
#ifndef RECURRENT_NN_AMD_H
#define RECURRENT_NN_AMD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rnn_status {
    RNN_OK = 0,
    RNN_ERR_INVALID_INPUT = 1,   /* bad attribute, shape, pointer or sequence length */
    RNN_ERR_UNSUPPORTED = 2,     /* valid, but beyond this library (scratch limit)   */
    RNN_ERR_DEVICE = 3,          /* a HIP call failed, or a device-side check fired  */
    RNN_ERR_OUT_OF_MEMORY = 4    /* host allocation failed                           */
} rnn_status;

typedef enum rnn_op { RNN_OP_RNN = 0, RNN_OP_GRU = 1, RNN_OP_LSTM = 2 } rnn_op;

/* Element type of the projection's operands.  BF16 rounds X and W to
 * bfloat16 (round to nearest even) and accumulates in float32; XW, the
 * recurrence, the states and the gate arithmetic stay float32. */
typedef enum rnn_proj_dtype { RNN_PROJ_F32 = 0, RNN_PROJ_BF16 = 1 } rnn_proj_dtype;

/* How the step loop is run.  AUTO picks PERSISTENT when every workgroup can be
 * resident at once, else PER_STEP. */
typedef enum rnn_kernel_path {
    RNN_PATH_AUTO = 0,
    RNN_PATH_PERSISTENT = 1,     /* one cooperative launch, device-wide step barrier */
    RNN_PATH_PER_STEP = 2        /* one launch per step (two for GRU lbr = 0)        */
} rnn_kernel_path;

/* Operator attributes (onemodel "Computation"/"Activations"; WebGPU README
 * "Attributes").  Zero-initialise and set what is needed. */
typedef struct rnn_attrs {
    int32_t op;                        /* rnn_op                                          */
    const char *direction;             /* "forward" | "reverse" | "bidirectional"; NULL = forward */
    int64_t hidden_size;               /* 0 = absent; else must equal R's last dimension  */
    int32_t layout;                    /* 0 or 1                                          */
    int32_t n_activations;             /* 0 = defaults (LSTM Sigmoid,Tanh,Tanh; GRU       */
    const char *const *activations;    /*   Sigmoid,Tanh; RNN Tanh); names case-insensitive;
                                          one set, or forward then reverse set            */
    int32_t n_alpha;                   /* activation_alpha, consumed in activation order  */
    const float *activation_alpha;
    int32_t n_beta;                    /* activation_beta, its own cursor                 */
    const float *activation_beta;
    int32_t has_clip;                  /* clamp pre-activations to [-clip, clip] only when */
    float clip;                        /*   has_clip && clip > 0; a NaN passes through    */
    int32_t input_forget;              /* LSTM only: forget gate = 1 - input gate         */
    int32_t linear_before_reset;       /* GRU only                                        */
    int32_t proj_dtype;                /* rnn_proj_dtype                                  */
    int32_t constant_weights;          /* W, R, B, P do not change between runs of this
                                          plan with this workspace: pack them once       */
    int32_t kernel_path;               /* rnn_kernel_path                                 */
    int32_t units_per_block;           /* 0 = automatic; hidden units per workgroup       */
    int32_t batch_tile;                /* 0 = automatic; batch rows per workgroup (16/32/64) */
    int32_t waves_per_block;           /* 0 = automatic; 4 or 8 waves split the step product */
    int32_t barrier_spin_limit;        /* 0 = default; polls before a step barrier gives up,
                                          raising the error rnn_workspace_check reports   */
    int32_t batch_halves;              /* 0 = automatic; 1 = each step over the whole batch
                                          tile; 2 = each step as two half-tile sub-steps, so
                                          that one half's H exchange overlaps the other
                                          half's product (needs R resident in registers, an
                                          RNN, LSTM or GRU with linear_before_reset = 1, and
                                          a batch tile of 32 or 64; else InvalidInput).
                                          Results are identical either way.              */
    int32_t time_chunk;                /* 0 = all steps at once; else steps per chunk: the
                                          projections and the H history are held for one
                                          chunk at a time and the states carry over between
                                          chunks, so the scratch limit applies to the chunk
                                          length instead of seq_length.  Results are
                                          identical either way.                          */
    int32_t exact;                     /* 1 = exact mode (onemodel "Exact mode"): every
                                          product value is one binary32 accumulator over
                                          k in increasing order from +0, each multiply and
                                          add rounded on its own (no matrix cores), and
                                          the transcendental activations follow one fixed
                                          binary64 method; results do not depend on the
                                          tiling and match that definition bit for bit.
                                          0 = fast mode (matrix-core products).           */
    int32_t fuse_projection;           /* 0 or 1 = the input projection as its own launch
                                          into a buffer of the workspace (the faster form
                                          where both apply); 2 = the projection inside the
                                          step loop, each workgroup computing the values of
                                          its own gate columns and rows one step ahead from
                                          its slice of W held in LDS, so that the workspace
                                          holds no projections (needs the two-half schedule
                                          in fast mode, an F32 projection, input_size a
                                          multiple of 256 and the slice within LDS; else
                                          InvalidInput).  Results are identical either way. */
} rnn_attrs;

/* Dimensions: hidden is R's last dimension, num_directions W's first. */
typedef struct rnn_dims {
    int64_t seq_length;
    int64_t batch_size;
    int64_t input_size;
    int64_t hidden;
    int64_t num_directions;
} rnn_dims;

typedef struct rnn_plan rnn_plan;

/*
 * rnn_plan_create -- validate attributes and dimensions, resolve the
 * activations (f, g, h per direction with alpha/beta cursors), choose the
 * tiling and lay out the workspace.  Host only: touches no device.
 *   attrs, dims: read during the call only.  *out receives a new plan.
 *   Errors, each with the passage that defines the rule (sections of the
 *   onemodel page "Recurrent operators: RNN, GRU, LSTM" unless stated):
 *   RNN_ERR_INVALID_INPUT for
 *     - an activation name outside the supported list, or a list that is
 *       neither one set nor (bidirectional) a forward and a reverse set
 *       .................................................. "Activations";
 *     - hidden 0, or a hidden_size attribute that differs from R's last
 *       dimension ....... "Choices the specification leaves open", hidden_size;
 *     - input_forget on a non-LSTM, linear_before_reset on a non-GRU (the
 *       attributes exist for those operators only) ......... "Computation";
 *     - layout other than 0 or 1 ..... "Choices ...", layout = 1; WebGPU README
 *       "Attributes";
 *     - an unknown op or direction, num_directions not matching direction
 *       (W's first dimension is the direction count) ..... WebGPU README
 *       "Inputs" and "Attributes";
 *     - negative sizes, time_chunk, barrier_spin_limit or tiling overrides
 *       outside their ranges (this library's own attributes);
 *   RNN_ERR_UNSUPPORTED when, per direction, L*batch*G*hidden + 4*batch*hidden
 *   (+ G*hidden*(input+hidden) unless constant_weights) reaches 2^30 floats,
 *   with L = seq_length, or the chunk length when time_chunk is set
 *   ............................................................... "Limits".
 */
rnn_status rnn_plan_create(const rnn_attrs *attrs, const rnn_dims *dims, rnn_plan **out);

/* Bytes of device workspace rnn_run needs for this plan (0 for zero-size). */
rnn_status rnn_plan_workspace_size(const rnn_plan *plan, size_t *bytes);

/*
 * rnn_run -- enqueue one operator invocation on `hip_stream` (a hipStream_t;
 * NULL = the null stream).  X, W, R are required; B, initial_h, initial_c, P
 * may be NULL (bias additions skipped, zero states, no peepholes);
 * sequence_lens may be NULL (every row runs seq steps) and is a HOST array of
 * batch_size int32 values in [0, seq].  Y, Y_h, Y_c may each be NULL (output
 * not wanted); Y_c, initial_c and P must be NULL unless the op is LSTM.
 * Y is written in full: positions t >= sequence_lens[b] hold +0.0; Y_h / Y_c
 * hold the state after each row's last valid step and 0 for a row of length
 * 0; with seq = 0 or batch = 0 they hold the initial states (or zeros).
 *   workspace: device memory of at least rnn_plan_workspace_size() bytes,
 *   256-byte aligned, owned by the caller, used by this run until the stream
 *   passes it.  With constant_weights the packed weights stay in it between
 *   runs: reuse the same workspace and weight pointers.
 *   Errors (nothing is enqueued): RNN_ERR_INVALID_INPUT for
 *     - a sequence length outside [0, seq] ..... "Choices the specification
 *       leaves open", sequence_lens (the run-time InvalidInput it names);
 *     - Y_c, initial_c or P given to a non-LSTM plan (LSTM-only tensors)
 *       ...................................... "Support"; WebGPU README "Inputs";
 *     - NULL X, W or R (required inputs) ........... WebGPU README "Inputs";
 *     - misaligned pointers or a workspace missing, too small or misaligned
 *       (this library's own conventions, above);
 *   RNN_ERR_DEVICE when a HIP call fails (the run may then be partial).
 */
rnn_status rnn_run(rnn_plan *plan, void *hip_stream, void *workspace, size_t workspace_bytes,
                   const float *X, const float *W, const float *R, const float *B,
                   const int32_t *sequence_lens, const float *initial_h,
                   const float *initial_c, const float *P,
                   float *Y, float *Y_h, float *Y_c);

/*
 * rnn_cell_run -- one step of the operator in the single-cell convention of
 * the OpenVINO page "RNNCell-3" (sections "Inputs" and "Outputs"; its formula
 * Ht = f(Xt Wi^T + Ht-1 Ri^T + Wbi + Rbi) in the description): the same
 * operator as rnn_run at seq_length 1, except that the bias is ONE vector,
 * the sum of the W and R biases, and only the new state is produced.
 *   plan: created with dims.seq_length = 1 and dims.num_directions = 1 (any
 *   op; the cell page itself defines the RNN cell, and the same convention is
 *   applied to GRU and LSTM gates).
 *   X [batch, input]; H [batch, hidden] (NULL = zeros); C [batch, hidden]
 *   (LSTM only, NULL = zeros); W [G*hidden, input]; R [G*hidden, hidden];
 *   B_sum [G*hidden] summed biases in the operator's gate order (NULL = no
 *   bias); P [3*hidden] (LSTM peepholes, NULL = none) -- all DEVICE pointers.
 *   H_out [batch, hidden] (required), C_out [batch, hidden] (LSTM only,
 *   nullable): the state after the step.  NaN is written as 0x7FC00000.
 *   The summed bias enters as ((X Wi^T + H Ri^T) + B_sum); internally it is
 *   the ONNX B with Wb = B_sum and Rb = +0, which is exact.  It is staged in
 *   the workspace, so the same workspace rules as rnn_run apply.
 *   Errors (nothing is enqueued): those of rnn_run, plus InvalidInput when
 *   the plan is not single-step and single-direction, when H_out is NULL, or
 *   when B_sum is given for GRU with linear_before_reset = 1 (its recurrent
 *   candidate bias is multiplied by the reset gate, so a sum cannot carry it:
 *   use rnn_run with the full B there).
 */
rnn_status rnn_cell_run(rnn_plan *plan, void *hip_stream, void *workspace, size_t workspace_bytes,
                        const float *X, const float *H, const float *C, const float *W,
                        const float *R, const float *B_sum, const float *P, float *H_out,
                        float *C_out);

/*
 * rnn_run_noalloc -- rnn_run for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same arguments without a workspace, the same launches and
 * results, and no allocating call at all.  Its scratch is a device array of
 * RNN_NOALLOC_SCRATCH_BYTES that the library holds on each GPU it runs on
 * until the process ends; sequence_lens reach the device as kernel arguments.
 *   Limits (RNN_ERR_UNSUPPORTED, nothing enqueued, no device call made): a plan
 *   whose rnn_plan_workspace_size() exceeds RNN_NOALLOC_SCRATCH_BYTES, or
 *   sequence_lens with more than RNN_NOALLOC_MAX_LENS_BATCH batch rows.
 *   Sharing: every call on one GPU uses that GPU's one scratch array, and each
 *   call leaves it holding its own state; calls that overlap in time on the
 *   same GPU (another stream, another thread, another plan) race and give
 *   undefined results.  Serialise them.  With constant_weights the packed
 *   weights are reused only while no other plan has run here in between.
 *   Stage timing (rnn_plan_enable_timing) records nothing on this path, and a
 *   barrier time-out is not reported (rnn_workspace_check needs a workspace).
 *   Other errors: those of rnn_run.
 */
#define RNN_NOALLOC_SCRATCH_BYTES (64u << 20)
#define RNN_NOALLOC_MAX_LENS_BATCH 256
rnn_status rnn_run_noalloc(rnn_plan *plan, void *hip_stream, const float *X, const float *W,
                           const float *R, const float *B, const int32_t *sequence_lens,
                           const float *initial_h, const float *initial_c, const float *P,
                           float *Y, float *Y_h, float *Y_c);

/*
 * rnn_workspace_check -- wait for `hip_stream`, then read the device-side
 * error word that the last run on this workspace left (a step barrier that
 * timed out).  RNN_OK when clean, RNN_ERR_DEVICE otherwise.  For tests of
 * this path, a plan created while the environment variable
 * RNN_AMD_TEST_WITHHOLD_FLAGS is set to a non-zero value never stores its
 * step flags, so every wait between steps runs out barrier_spin_limit (results
 * are then undefined, and the kernel still finishes).
 */
rnn_status rnn_workspace_check(const rnn_plan *plan, void *hip_stream, const void *workspace);

/*
 * rnn_plan_enable_timing -- when enabled, rnn_run records HIP events around
 * each stage on its stream; rnn_plan_last_timings then waits for them and
 * writes up to n durations in milliseconds of the last run, in the order
 * pack, projection, recurrence, other (init and final writes).
 */
rnn_status rnn_plan_enable_timing(rnn_plan *plan, int32_t enable);
rnn_status rnn_plan_last_timings(rnn_plan *plan, float *ms, int32_t n);

/* A short human-readable description of the tiling and kernel path. */
rnn_status rnn_plan_describe(const rnn_plan *plan, char *buf, size_t len);

/* Release a plan (host memory only).  NULL is a no-op. */
void rnn_plan_destroy(rnn_plan *plan);

/* ------------------------------------------------------------------------
 * Operators of a selective-state language model: the layer whose recurrence is
 * linear with coefficients that depend on the input, its short convolution,
 * its projections in 8-bit integers, and the scores of what it answers.
 *
 * Conventions, besides those above
 *   - No plan: a descriptor of sizes, strides and types goes with each call and
 *     is read during it.  Strides count elements; the last dimension of every
 *     tensor is contiguous.  Tensors need the alignment of their elements only
 *     (rows whose base and strides are multiples of 16 bytes run faster).
 *   - sequence_lens is a DEVICE int32 array here, so that a serving loop can
 *     keep lengths where it computes them and a captured graph can be replayed
 *     with others; values outside [0, steps] are taken as the nearest of the
 *     two.  Positions t >= sequence_lens[b] are not read, and their outputs
 *     are +0.0.
 *   - A state of a row of length 0 (or of a call with steps = 0) is handed on
 *     as it came; state_out may be state_in (in place), no other output may
 *     overlap an input.
 *   - Sums, states and exponentials are float32 whatever the tensors' type, and
 *     rounded once (to nearest even) where a value is stored in fewer bits.
 *   - A launch has fewer than 2^32 threads; what would need more is
 *     RNN_ERR_UNSUPPORTED, and nothing is enqueued.
 *   - Every call is stream-ordered, allocates nothing and may be captured.
 *     Nothing is kept between calls.  Workspaces: device memory, 256-byte
 *     aligned, of at least the bytes that the matching *_workspace_size
 *     gives, in use until the stream passes the call.
 * ---------------------------------------------------------------------- */

/* Element types of the tensors below. */
typedef enum rnn_dtype {
    RNN_DTYPE_F32 = 0,
    RNN_DTYPE_BF16 = 1,
    RNN_DTYPE_F16 = 2,
    RNN_DTYPE_I8 = 3
} rnn_dtype;

#define RNN_CONV_MAX_TAPS 8
#define RNN_SCAN_MAX_STATES 64
#define RNN_QUANT_MAX_COLS 131071
#define RNN_SCORES_MAX_TOP 64

/* x and y [batch, steps, dim]; weight [dim, taps], bias [dim] float32;
 * states [batch, taps - 1, dim] dense, of x's type. */
typedef struct rnn_conv_desc {
    int64_t batch, steps, dim;
    int64_t x_batch_stride, x_step_stride;
    int64_t y_batch_stride, y_step_stride;
    int32_t taps;                      /* 1 to RNN_CONV_MAX_TAPS                      */
    int32_t silu;                      /* 1: y = v / (1 + exp(-v)) of the sum v       */
    int32_t dtype;                     /* of x, y and the states: F32, BF16 or F16    */
} rnn_conv_desc;

/*
 * rnn_conv_run -- causal convolution of each channel over the last `taps`
 * steps:  v[b,t,c] = bias[c] + sum_{j < taps} weight[c,j] xx[b, t + j, c], where
 * xx is state_in (the taps - 1 inputs before the first step, oldest first; NULL
 * = zeros) followed by x.  state_out (nullable) receives the taps - 1 inputs
 * before step sequence_lens[b].  One new token is a call with steps = 1.
 *   bias, state_in, sequence_lens, state_out may be NULL.
 *   Errors (nothing is enqueued): RNN_ERR_INVALID_INPUT for sizes below 0, taps
 *   or dtype outside their ranges, a missing or misaligned tensor, y on x;
 *   RNN_ERR_UNSUPPORTED for 2^32 or more threads (one takes 8 bytes of channels,
 *   or one channel, and 8 to 32 steps).
 */
rnn_status rnn_conv_run(const rnn_conv_desc *desc, void *hip_stream, const void *x,
                        const float *weight, const float *bias, const void *state_in,
                        const int32_t *sequence_lens, void *y, void *state_out);

/* x, dt, z, y [batch, steps, dim]; B, C [batch, steps, groups, states];
 * A [dim, states], D and dt_bias [dim] float32; states [batch, dim, states]
 * float32, dense. */
typedef struct rnn_scan_desc {
    int64_t batch, steps, dim, states, groups;   /* channel c reads group c / (dim / groups) */
    int64_t x_batch_stride, x_step_stride;
    int64_t dt_batch_stride, dt_step_stride;
    int64_t z_batch_stride, z_step_stride;
    int64_t y_batch_stride, y_step_stride;
    int64_t B_batch_stride, B_step_stride, B_group_stride;
    int64_t C_batch_stride, C_step_stride, C_group_stride;
    int32_t dtype;                     /* of x, dt, z, y, B and C: F32, BF16 or F16   */
    int32_t dt_softplus;               /* 1: step sizes log(1 + exp(dt + dt_bias))    */
} rnn_scan_desc;

/*
 * rnn_scan_run -- selective state space scan.  With the step size
 * s = dt[b,t,c] + dt_bias[c] (through log(1 + exp(.)) with dt_softplus), for
 * every channel c and state n, t = 0, 1, ...:
 *     h[n] = exp(s A[c,n]) h[n] + s x[b,t,c] B[b,t,g,n]
 *     y[b,t,c] = (sum_n C[b,t,g,n] h[n] + D[c] x[b,t,c]) * z / (1 + exp(-z))
 * with h = state_in (NULL = zeros) before the first step and state_out
 * (nullable) = h after the last one.  One new token is a call with steps = 1.
 *   D (no skip), z (no gate), dt_bias, state_in, sequence_lens, state_out may
 *   be NULL.  A is taken as given (negative for a state that decays).
 *   Errors (nothing is enqueued): RNN_ERR_INVALID_INPUT for sizes below 0,
 *   states outside 1 to RNN_SCAN_MAX_STATES, groups that do not divide dim,
 *   an unknown dtype, a missing or misaligned tensor, y on an input, a
 *   workspace missing, too small or misaligned; RNN_ERR_UNSUPPORTED for more
 *   than 2^31 - 1 channels or steps, or 2^32 or more threads: up to 8 to 64 steps
 *   (by the sizes) a quarter of the states has one, beyond that 16 channels have
 *   512 in each span of the steps.
 */
rnn_status rnn_scan_workspace_size(const rnn_scan_desc *desc, size_t *bytes);
rnn_status rnn_scan_run(const rnn_scan_desc *desc, void *hip_stream, void *workspace,
                        size_t workspace_bytes, const void *x, const void *dt, const float *A,
                        const void *B, const void *C, const float *D, const void *z,
                        const float *dt_bias, const float *state_in,
                        const int32_t *sequence_lens, void *y, float *state_out);

/*
 * rnn_quantize_rows -- rows of x [rows, cols] to 8-bit integers with one scale
 * each:  m = max |x|, r = 127 / m, q = x r rounded to the nearest even integer,
 * scale = m / 127, each operation rounded to float32.  A row with m < 2^-100
 * gives q = 0 and scale 0; one that holds an infinity or a NaN gives q = 0 and
 * scale NaN.  q is [rows, q_stride] with q_stride >= cols a multiple of 16 bytes,
 * 16-byte aligned; columns from cols to q_stride are written as 0.
 *   The weights of rnn_quant_project are rounded by it once (a row is an output
 *   channel), activations that several projections share once for each token.
 *   Errors: RNN_ERR_INVALID_INPUT for sizes below 0, strides or dtype outside
 *   their ranges, a missing or misaligned tensor; RNN_ERR_UNSUPPORTED for
 *   2^31 rows or more, a q_stride above 2^30, or 2^32 or more threads (4, 16, 64,
 *   256 or 1024 a row: up to 128, 512, 2048, 32768 or more columns).
 */
rnn_status rnn_quantize_rows(void *hip_stream, int64_t rows, int64_t cols, int32_t dtype,
                             const void *x, int64_t x_stride, int8_t *q, int64_t q_stride,
                             float *scale);

typedef struct rnn_quant_desc {
    int64_t rows, cols, outs;          /* y [rows, outs] = x [rows, cols] . w [outs, cols]^T */
    int64_t x_stride, w_stride, y_stride;
    int32_t x_dtype;                   /* F32, BF16, F16: rounded to 8 bits in the call by
                                          the rule of rnn_quantize_rows; I8: already are   */
    int32_t y_dtype;                   /* F32, BF16 or F16                             */
} rnn_quant_desc;

/*
 * rnn_quant_project -- y[i,o] = (sum_k qx[i,k] w[o,k]) * (x_scale[i] * w_scale[o])
 * + bias[o], the sum exact in 32-bit integers.  w is int8 [outs, w_stride]: base
 * and w_stride multiples of 16 bytes, every row readable up to `cols` rounded up
 * to 16 (the columns past `cols` may hold anything).  With x_dtype I8, x follows
 * the same rule and x_scale [rows] is required; else x_scale must be NULL.  bias [outs]
 * float32 may be NULL.
 *   Errors (nothing is enqueued): RNN_ERR_INVALID_INPUT for sizes below 0,
 *   strides or types outside their ranges, a missing or misaligned tensor, a
 *   workspace missing, too small or misaligned; RNN_ERR_UNSUPPORTED for cols
 *   above RNN_QUANT_MAX_COLS (beyond it a 32-bit sum can overflow), for
 *   2^31 - 2^16 rows or outs or more, or for 2^32 or more threads (up to 16 rows,
 *   16 an output; beyond that 512 a tile of 256 x 256; those of rnn_quantize_rows).
 */
rnn_status rnn_quant_workspace_size(const rnn_quant_desc *desc, size_t *bytes);
rnn_status rnn_quant_project(const rnn_quant_desc *desc, void *hip_stream, void *workspace,
                             size_t workspace_bytes, const void *x, const float *x_scale,
                             const int8_t *w, const float *w_scale, const float *bias, void *y);

typedef struct rnn_scores_desc {
    int64_t rows, vocab;               /* logits [rows, vocab]                         */
    int64_t logits_stride;
    int32_t dtype;                     /* of the logits: F32, BF16 or F16              */
    int32_t token_bytes;               /* tokens are int32 (4) or int64 (8)            */
    int32_t top;                       /* alternatives, 0 to RNN_SCORES_MAX_TOP        */
} rnn_scores_desc;

/*
 * rnn_token_scores -- what a row of logits x says of a token k, with
 * p_v = exp(x_v) / sum_u exp(x_u):  logprob = log p_k;  entropy = -sum p_v log p_v
 * (0 log 0 = 0);  rank = the number of entries before the token in decreasing
 * order of x, equal ones in increasing order of their index;  the first `top`
 * entries of that order as log probabilities (top_logprobs [rows, top]) and
 * indices (top_ids [rows, top]).  -0 and +0 are equal, NaN is before every number.
 *   tokens is a DEVICE array [rows]; a token outside [0, vocab) has logprob NaN
 *   and rank -1 (its row's other outputs are computed).  A row of -inf only, or
 *   one that holds +inf or NaN, has no distribution: its logprobs and entropy
 *   are NaN, its rank and top_ids follow the order above.  Where top > vocab the
 *   rest of top_ids is -1 and of top_logprobs -inf.
 *   tokens may be NULL if logprob and rank are; any output may be NULL.
 *   Errors (nothing is enqueued): RNN_ERR_INVALID_INPUT for sizes below 0, top,
 *   dtype, token_bytes or stride outside their ranges, a missing or misaligned
 *   tensor, a workspace missing, too small or misaligned; RNN_ERR_UNSUPPORTED
 *   for 2^31 rows, a vocabulary of 2^31 - 2^16 or more, or 2^32 or more threads
 *   (64 a row up to 2048 entries, 256 beyond).
 */
rnn_status rnn_scores_workspace_size(const rnn_scores_desc *desc, size_t *bytes);
rnn_status rnn_token_scores(const rnn_scores_desc *desc, void *hip_stream, void *workspace,
                            size_t workspace_bytes, const void *logits, const void *tokens,
                            float *logprob, float *entropy, int32_t *rank,
                            float *top_logprobs, int32_t *top_ids);

/* Thread-local text describing the last non-OK status on this thread. */
const char *rnn_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* RECURRENT_NN_AMD_H */
