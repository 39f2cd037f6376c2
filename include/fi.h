/*
 * fi.h -- exact online causal long convolution on AMD MI355X (gfx950).
 *
 * Citations name the web page "Flash Inference: Inferenza in Tempo
 * Quasi-Lineare per Modelli di Sequenza a Convoluzione Lunga e Oltre"
 * (lowest.today summary of arXiv 2410.12982), written [FI], and its sections.
 *
 * The operation ([FI] "Definizione del Compito", "Definizione Specifica di
 * LCSM"), 0-indexed: for every channel (b, c), b in [0,B), c in [0,D),
 *
 *     y[b][t][c] = sum_{s=0}^{t} h[t-s][c] * x[b][s][c],     t in [0, L),
 *
 * where x[b][t+1][.] may only be supplied after y[b][t][.] has been returned
 * (online constraint).  The filter h[L][D] is shared by the B batch rows.  The
 * library evaluates it with the relaxed power-of-two tiling of [FI]
 * "Strategia di Tiling (Algoritmo 1)": once position i-1 is complete, with
 * U = largest power of two dividing i, the tile tau(x, [i-U, i), h, [i, i+U))
 * of [FI] "Definizione di Aggregazione di Contribuzione" adds the contribution
 * of x[i-U, i) to y[i, i+U) (clipped to < L).  Small tiles are direct
 * Toeplitz products, larger ones FFT circular convolutions of length 2U with
 * precomputed filter spectra ([FI] "Ottimizzazione della Memoria", "Trucco
 * di Convoluzione Circolare").  fi_step does tiles of side U <= T (the
 * config's small_tile_max) directly; the persistent pass (fi_run_closed_loop,
 * fi_run_prompted) does every tile of side < 256 and, for T < 256, the tile
 * of side 256 directly (on the matrix cores), and the larger ones by FFT.
 * The results agree to fp32 rounding.
 *
 * Layouts: row-major, channels innermost: h[L][D], x[B][L][D], y[B][L][D],
 * per-step vectors [B][D].  Storage dtype of x and h is the config's io_dtype
 * (fp32 or bf16); y is always fp32 and all arithmetic is fp32.
 *
 * Pointers: every array argument is a DEVICE pointer (hipMalloc'ed or a
 * torch CUDA tensor's data_ptr()) unless stated.  Calls other than
 * fi_create / fi_destroy are asynchronous on the config's stream: the caller
 * owns its arrays and must keep them valid until that stream is synchronised.
 *
 * Errors: functions return FI_OK (0) or a negative FI_ERR_* code and never
 * throw.  Arguments are validated before any device work; a rejected call
 * changes nothing.  FI_ERR_HIP records the HIP error, readable through
 * fi_strerror(FI_ERR_HIP) on the same thread.  A handle is not thread-safe;
 * distinct handles are independent.
 */
#ifndef FI_H_
#define FI_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct fi_handle fi_handle;  /* opaque; owns all the device memory it allocates */

/* Storage type of x and h (y and every accumulation are always fp32). */
typedef enum { FI_F32 = 0, FI_BF16 = 1 } fi_dtype;

/* Feedback of fi_run_closed_loop. */
typedef enum {
    FI_FEEDBACK_NONE = 0,   /* open loop: x[b][t][c] read from x_in[B][L][D] */
    FI_FEEDBACK_TANH = 1    /* closed loop: x[b][t+1][c] = tanh(y[b][t][c]) */
} fi_feedback;

enum {
    FI_OK = 0,
    FI_ERR_INVALID = -1,      /* bad argument: NULL, size <= 0, overflow, unknown enum */
    FI_ERR_NOMEM = -2,        /* device allocation failed */
    FI_ERR_HIP = -3,          /* HIP runtime error (see fi_strerror) */
    FI_ERR_STATE = -4,        /* call not allowed at the handle's current position */
    FI_ERR_UNSUPPORTED = -5   /* valid but not supported (e.g. no gfx950 device) */
};

/* largest supported L (fi_create returns FI_ERR_UNSUPPORTED beyond it) */
#define FI_MAX_L (1LL << 25)

/* small_tile_max used when the config leaves it 0 */
#define FI_DEFAULT_SMALL_TILE_MAX 64

typedef struct {
    int64_t B;               /* batch rows, >= 1 */
    int64_t D;               /* channels per row, >= 1 */
    int64_t L;               /* positions = filter length, >= 1 (any value; tiles clip to < L) */
    fi_dtype io_dtype;       /* FI_F32 or FI_BF16 (an int-sized enum) */
    void *stream;            /* hipStream_t the handle works on; NULL = the null stream */
    int32_t small_tile_max;  /* T: the largest tile side fi_step does as a direct product, tiles of
                                side > T being FFT tiles: 64, 128 or 256; 0 = the environment's
                                FI_SMALL_TILE_MAX when set (an override for ablations; any other
                                value there gives FI_ERR_INVALID), else FI_DEFAULT_SMALL_TILE_MAX.  The persistent pass (fi_run_closed_loop,
                                fi_run_prompted) does every tile of side < 256 directly whatever T
                                is; it does the tile of side 256 from LDS when T = 256, else on
                                the matrix cores, and the larger ones by FFT. */
} fi_config;

/*
 * fi_create: validate cfg, allocate the handle's device state, copy the
 * filter h[L][D] (device pointer, io_dtype) and precompute, on the device,
 * the filter spectra of every FFT tile level ([FI] "Ottimizzazione della
 * Memoria": the filter DFT is computed ahead for each block size) and the
 * twiddle tables.  Synchronous: returns after the device work finished, so
 * the caller may free h at once.  On success *out receives the handle at
 * position 0; on failure *out is set to NULL and nothing stays allocated.
 * Errors: FI_ERR_INVALID for a NULL pointer, B, D or L < 1, an unknown dtype
 * or small_tile_max, or sizes whose element counts overflow; FI_ERR_UNSUPPORTED
 * for L > FI_MAX_L or when the current device is not gfx950; FI_ERR_NOMEM /
 * FI_ERR_HIP from the device.
 */
int fi_create(const fi_config *cfg, const void *h, fi_handle **out);

/*
 * fi_step: one online step at the handle's position t ([FI] "Strategia di
 * Tiling (Algoritmo 1)", one loop iteration): reads x_t[B][D] (io_dtype),
 * writes y_t[B][D] (fp32) = accumulated tiles + h[0] * x_t (the red cell),
 * then, if t+1 < L, applies the tile of side lowbit(t+1).  Position becomes
 * t+1.  FI_ERR_STATE when the position already is L.
 */
int fi_step(fi_handle *s, const void *x_t, float *y_t);

/*
 * fi_run_closed_loop: all L steps in one call, from position 0 (else
 * FI_ERR_STATE); leaves the position at L.  One persistent device pass: a
 * single kernel launch on the handle's stream, which may be captured into a
 * HIP graph and replayed (the pass clears the state it uses itself; the
 * handle's position is host state and is not replayed).
 *   fb = FI_FEEDBACK_TANH: x_in is x_0[B][D]; x[t+1] = tanh(y[t]) (rounded to
 *        bf16, nearest-even, when io_dtype is FI_BF16).
 *   fb = FI_FEEDBACK_NONE: x_in is x[B][L][D] (the open-loop inputs, consumed
 *        in order through the same online schedule).
 *   y[B][L][D] (fp32) receives every output; x_out[B][L][D] (io_dtype), if not
 *   NULL, receives the inputs that produced them.
 */
int fi_run_closed_loop(fi_handle *s, const void *x_in, fi_feedback fb, float *y, void *x_out);

/*
 * fi_run_prompted: generation from a prompt ([FI] "Definizione del Compito":
 * the prompt x_1 .. x_p is given, later inputs are produced one by one), all
 * L steps in one call from position 0 (else FI_ERR_STATE), leaving the
 * position at L.  Positions t < p read x_prompt[B][p][D] (io_dtype); from
 * position p on, x[t] = tanh(y[t-1]) (rounded to bf16, nearest-even, when
 * io_dtype is FI_BF16).  Every output goes through the same online schedule
 * as fi_run_closed_loop; p = 1 is its closed loop with x_0 = x_prompt[.][0][.]
 * and p = L its open loop.  y[B][L][D] (fp32) receives every output; x_out
 * [B][L][D] (io_dtype), if not NULL, the inputs that produced them (the
 * prompt's values unchanged).  FI_ERR_INVALID for a NULL handle, x_prompt or
 * y, or p outside [1, L].  The caller owns x_prompt, y and x_out, which must
 * stay valid until the stream has passed the call.
 */
int fi_run_prompted(fi_handle *s, const void *x_prompt, int64_t p, float *y, void *x_out);

/*
 * fi_conv_static: for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * fi_create + fi_run_closed_loop + fi_destroy in one call that allocates
 * nothing.  Same arguments and results as those calls: cfg, h[L][D]
 * (io_dtype) as for fi_create; x_in, fb, y, x_out as for fi_run_closed_loop.
 * The handle's device buffers (filter rows, accumulator rows, spectra,
 * twiddles, FFT scratch) are carved from one fixed workspace of
 * FI_STATIC_WORKSPACE_BYTES per device, a static device array the library
 * holds until the process ends; no hipMalloc, hipFree or other allocating
 * call is made.  Their size is about 4 LS (D + B D) + 8 D L bytes (LS = L
 * rounded up to 64) plus twiddle tables and, when L > 8192, FFT scratch of
 * 8 * min(B D, resident teams) * (largest tile side) bytes; larger problems
 * get FI_ERR_UNSUPPORTED and nothing is launched.  Asynchronous on
 * cfg->stream (nothing is synchronised): the caller keeps h, x_in, y and
 * x_out valid until the stream has passed the call.  Every call on a device
 * uses that device's one workspace: calls that overlap on one device (on
 * different streams, or from different threads) race and give undefined
 * results; calls in order on one stream are safe.  Errors as fi_create and
 * fi_run_closed_loop (FI_ERR_INVALID, FI_ERR_UNSUPPORTED, FI_ERR_HIP).
 */
#define FI_STATIC_WORKSPACE_BYTES (64LL << 20)
int fi_conv_static(const fi_config *cfg, const void *h, const void *x_in, fi_feedback fb, float *y,
                   void *x_out);

/*
 * The layer stack ([FI] "Algoritmo di Inferenza LCSM (Algoritmo 2)",
 * "Parallelizzazione Cross-Layer (Algoritmo 3)"): M layers, each a long
 * convolution mixer (filter rho^l[L][D], per channel) followed by a block
 * (the synthetic MLP + GELU block of [FI] "Configurazione Sperimentale"),
 * and a sampler that feeds the last layer's output back with added noise.
 * 0-indexed, for every batch row b and position t, with a^0 = x:
 *   z^l_t[c]  = sum_{s<=t} rho^l[t-s][c] a^l_s[c]
 *   a^{l+1}_t = W2^l act(W1^l z^l_t)          (W row j = output j, D x D)
 *   x_{t+1}   = a^M_t + sigma noise[t]
 * The mixers run the relaxed tiling of fi_step on all M B D channels (red
 * cells and blocks of all layers in order at each position, then the gray
 * tiles of all layers in one launch).  fp32 storage and arithmetic.
 */
typedef struct fi_stack fi_stack;   /* opaque; owns its device memory */
typedef enum { FI_ACT_GELU = 0, FI_ACT_TANH = 1, FI_ACT_IDENTITY = 2 } fi_activation;
typedef struct {
    int64_t B;                /* batch rows, >= 1 */
    int64_t D;                /* channels (the blocks are D x D), 1 <= D <= 8192 */
    int64_t L;                /* positions = filter length, >= 1 */
    int64_t M;                /* layers, >= 1 */
    fi_activation act;        /* the blocks' activation: GELU (exact, erf), tanh or identity */
    void *stream;             /* hipStream_t; NULL = the null stream */
    int32_t small_tile_max;   /* T as in fi_config (0 = default) */
} fi_stack_config;

/* fi_stack_create: copies rho[M][L][D], w1[M][D][D] and w2[M][D][D] (device
 * pointers, fp32; W[l][j][k] is the weight of input k in output j) and
 * precomputes every layer's filter spectra.  Synchronous.  Errors as
 * fi_create (FI_ERR_INVALID for an unknown act or M < 1;
 * FI_ERR_UNSUPPORTED for D > 8192). */
int fi_stack_create(const fi_stack_config *cfg, const float *rho, const float *w1, const float *w2,
                    fi_stack **out);

/* fi_stack_run: generates all L positions from x0[B][D]: y[B][L][D]
 * receives a^M_t, x_out[B][L][D] (or NULL) the inputs x_t; noise[B][L][D]
 * (or NULL: no noise) is scaled by sigma.  Each call starts from position 0.
 * It first waits for the stream to pass the handle's earlier runs, then
 * queues one launch per position (two where the position completes a tile
 * of side > 16) and returns: device pointers, owned by the caller until the
 * stream has passed the call.  A position's layers run on up to 16
 * workgroups that wait for each other's partial products; a wait past its
 * limit (about a second: the workgroups could not all be resident) leaves
 * garbage in that run's outputs and makes this and every later call on the
 * handle return FI_ERR_HIP.  L M must not exceed 2^30 (FI_ERR_UNSUPPORTED
 * at fi_stack_create). */
int fi_stack_run(fi_stack *s, const float *x0, const float *noise, float sigma, float *y, float *x_out);

/* fi_stack_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_stack_destroy(fi_stack *s);

/* fi_reset: position := 0; the accumulators are cleared on the stream before
 * the next fi_step (fi_run_closed_loop clears the rows it uses itself). */
int fi_reset(fi_handle *s);

/* fi_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_destroy(fi_handle *s);

/* fi_position: the handle's current position (host value), or -1 for NULL. */
int64_t fi_position(const fi_handle *s);

/* fi_strerror: static description of a status code (host; thread-local text
 * for FI_ERR_HIP includes the last HIP error seen on this thread). */
const char *fi_strerror(int status);

/*
 * Schedule helper (host, integer only): the tile applied once position i-1
 * is complete, for 1 <= i < L ([FI] "Strategia di Tiling (Algoritmo 1)",
 * "Analisi di Complessita (Proposizione 1)"): U = largest power of two dividing
 * i, inputs [in_lo, in_hi) = [i-U, i), outputs [out_lo, out_hi) =
 * [i, min(i+U, L)).  FI_ERR_INVALID for i outside [1, L) or a NULL out.
 */
typedef struct {
    int64_t U, in_lo, in_hi, out_lo, out_hi;
} fi_tile;
int fi_tile_at(int64_t L, int64_t i, fi_tile *out);

/*
 * Operators around the mixers: what a decoder that mixes long convolutions
 * with linear attention runs between and after them.  They stand beside the
 * convolution and use the same conventions: device pointers, asynchronous on
 * the config's stream, FI_* status codes, arguments checked before any device
 * work, and nothing allocated after the create calls.  A handle's calls share
 * its workspace, so they are made in order on its one stream.
 *
 * An array of positions is given as a view: element c of head h at position t
 * of row b lies at p + b*row + t*pos + h*head + c (strides counted in
 * elements; any value, 0 broadcasts an input).  Elements of a head are
 * adjacent.  The values do not depend on strides and alignment; aligned views
 * (p, strides and head sizes in multiples of 16 bytes) load faster.
 */
typedef struct {
    void *p;              /* aligned to its element */
    int64_t row, pos, head;
} fi_view;

/*
 * Linear attention with a decay per head.  For every row b, key/value head n
 * and position t, with lam_n = exp(log_decay[n]) in [0, 1]:
 *
 *     S[t] = lam_n S[t-1] + k[t] v[t]^T           (S is dk x dv)
 *     o[t][h] = scale * S[t]^T q[t][h]            for the H/Hkv query heads h of
 *                                                 group n (h / (H/Hkv) == n)
 *
 * q, k, v and o are of io_dtype; S is held, summed and stored in fp32, and o
 * is rounded to io_dtype once.  (bf16 prompts: the fp32 factors of the matrix
 * products, S and the weights of the values, enter as two bf16 parts each, which
 * hold them to 2^-16.)  A state array is state[n_slots][Hkv][dk][dv] (fp32, dense, the caller's); row
 * b uses slot slots[b], or slot b where slots is NULL.  A row whose slot is
 * outside [0, n_slots) takes no part: its o is zero and no state changes.
 * Two rows of one call must not share a slot (their updates would race).
 */
typedef struct fi_lattn fi_lattn;   /* opaque; owns its device memory */
typedef struct {
    int64_t B;                /* most rows of one call, >= 1 */
    int64_t L;                /* most positions of one fi_lattn_prompt call, >= 1 */
    int64_t H;                /* query heads, a multiple of Hkv */
    int64_t Hkv;              /* key/value heads, >= 1 */
    int64_t dk, dv;           /* sizes of a key and of a value head, 1 .. 256 */
    float scale;              /* multiplies o; finite */
    fi_dtype io_dtype;        /* type of q, k, v and o */
    void *stream;             /* hipStream_t; NULL = the null stream */
} fi_lattn_config;

typedef struct {
    int64_t B, L;             /* rows and positions of this call, within the config's */
    fi_view q, k, v;          /* [B][L][H][dk], [B][L][Hkv][dk], [B][L][Hkv][dv] */
    fi_view o;                /* [B][L][H][dv]; overlaps no input */
    const int32_t *lens;      /* [B] on the device: row b has lens[b] positions (taken into [0, L]); NULL:
                                 all have L.  What lies past a row's end is not read as a number; o is zero there. */
    const int32_t *slots;     /* [B] on the device, or NULL */
    int64_t n_slots;          /* states in `state` (>= B where slots is NULL) */
    float *state;             /* read and updated in place, aligned to 16 bytes; may be NULL in a fresh prompt */
    int32_t fresh;            /* nonzero: every row begins from S = 0, whatever its slot holds */
} fi_lattn_args;

/* fi_lattn_create: copies log_decay[Hkv] (device, fp32; each <= 0, -inf for
 * lam = 0) and allocates the workspace of the longest prompt.  Synchronous.
 * FI_ERR_INVALID for a NULL pointer, a size < 1, H not a multiple of Hkv, a
 * NaN or positive log_decay, an infinite or NaN scale, an unknown dtype or
 * sizes that overflow; FI_ERR_UNSUPPORTED for dk or dv > 256, L > FI_MAX_L,
 * B Hkv > 2^20 or a device that is not gfx950; FI_ERR_NOMEM / FI_ERR_HIP from the device. */
int fi_lattn_create(const fi_lattn_config *cfg, const float *log_decay, fi_lattn **out);

/* fi_lattn_prompt: L given positions of every row in the chunked form (matrix
 * products over chunks of positions; one position with states: the recurrent
 * form), from the row's state, which is left after its last position.  B = 0 and L = 0 are allowed.  FI_ERR_INVALID for
 * a NULL pointer, sizes beyond the config's, fewer than B states without
 * slots, or a pointer that is not aligned to its element.  A NaN or infinity
 * in k or v at t makes every later output and the state not finite, and can
 * make outputs of up to 63 positions before t of its row and head NaN. */
int fi_lattn_prompt(fi_lattn *s, const fi_lattn_args *a);

/* fi_lattn_step: one new position of every row in the recurrent form; L is 1,
 * lens NULL and state not NULL, also where fresh (else FI_ERR_INVALID).  Errors
 * as fi_lattn_prompt. */
int fi_lattn_step(fi_lattn *s, const fi_lattn_args *a);

/* fi_lattn_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_lattn_destroy(fi_lattn *s);

/*
 * Dense product with its epilogue, for any number of rows:
 *
 *     y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + res[m][n]
 *
 * x[M][K], w[N][K] (row n = output n, as the stack's blocks) and bias[N] are
 * of io_dtype, res and y of out_dtype; sums are fp32 (fp32 storage: fp32
 * products), rounded once.  Rows are ld* elements apart.
 */
typedef struct fi_dense fi_dense;   /* opaque; owns its device memory */
typedef struct {
    int64_t M;                /* most rows of one call, >= 1 */
    int64_t N, K;             /* outputs and inputs of a row, >= 1 */
    fi_dtype io_dtype, out_dtype;
    fi_activation act;
    void *stream;             /* hipStream_t; NULL = the null stream */
} fi_dense_config;
typedef struct {
    int64_t M;                /* rows of this call, 0 .. the config's */
    const void *x; int64_t ldx;
    const void *w; int64_t ldw;
    const void *bias;         /* or NULL */
    const void *res; int64_t ldr;   /* res or NULL; res = y with ldr = ldy adds in place */
    void *y; int64_t ldy;     /* overlaps no other input */
} fi_dense_args;

/* fi_dense_create: allocates the workspace.  FI_ERR_INVALID for a NULL
 * pointer, a size < 1 or beyond 2^31 - 1, an unknown dtype or activation;
 * FI_ERR_UNSUPPORTED for M or N > 2^27 or when the device is not gfx950;
 * FI_ERR_NOMEM / FI_ERR_HIP from the device. */
int fi_dense_create(const fi_dense_config *cfg, fi_dense **out);

/* fi_dense_run: FI_ERR_INVALID for a NULL pointer, M beyond the config's, a
 * row stride below the row's length (ldx, ldw >= K; ldr, ldy >= N), or a
 * pointer that is not aligned to its element. */
int fi_dense_run(fi_dense *s, const fi_dense_args *a);

/* fi_dense_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_dense_destroy(fi_dense *s);

/*
 * Token scores: per row of logits z[V] (times `scale`, 1/temperature), with
 * p = softmax(scale z) in fp32,
 *
 *     lse = log sum_j exp(scale z[j]),   logprob = scale z[target] - lse,
 *     entropy = -sum_j p[j] log p[j],
 *     top[0..k), top_id[0..k): the k most probable tokens, log probability and
 *         index, most probable first, ties to the lowest index.
 *
 * A logit of -inf is a token that a mask rules out: it adds nothing, its log
 * probability is -inf and it is no alternative; where fewer than k tokens are
 * left, the further entries are -1 and -inf.  A row without any token has lse
 * and logprob -inf and entropy 0.  A row with a NaN or +inf has NaN in lse,
 * logprob, entropy and top, and -1 in top_id.  A target < 0 asks for nothing
 * (logprob 0); one >= V gives NaN.
 */
typedef struct fi_scores fi_scores;   /* opaque; owns its device memory */
#define FI_SCORES_MAX_K 32
typedef struct {
    int64_t rows;             /* most rows of one call, >= 1 */
    int64_t V;                /* tokens of the vocabulary, 1 .. 2^31 - 1 */
    int32_t k;                /* alternatives per row, 0 .. FI_SCORES_MAX_K */
    fi_dtype io_dtype;        /* type of the logits */
    float scale;              /* finite, > 0 */
    void *stream;             /* hipStream_t; NULL = the null stream */
} fi_scores_config;
typedef struct {
    int64_t rows;             /* rows of this call, 0 .. the config's */
    const void *logits; int64_t ld;   /* rows ld >= V elements apart */
    const int64_t *targets;   /* [rows], or NULL (then logprob is NULL too) */
    float *logprob, *entropy, *lse;   /* [rows] each; each may be NULL */
    float *top;               /* [rows][k]; NULL where k = 0 */
    int64_t *top_id;          /* [rows][k]; NULL where k = 0 */
} fi_scores_args;

/* fi_scores_create: allocates the workspace.  FI_ERR_INVALID for a NULL
 * pointer, a size, k or scale out of range or an unknown dtype;
 * FI_ERR_UNSUPPORTED when the device is not gfx950; FI_ERR_NOMEM / FI_ERR_HIP
 * from the device. */
int fi_scores_create(const fi_scores_config *cfg, fi_scores **out);

/* fi_scores_run: FI_ERR_INVALID for a NULL handle, args or logits, rows beyond
 * the config's, ld < V, logprob without targets (or targets without logprob),
 * top or top_id NULL where k > 0, or a pointer not aligned to its element. */
int fi_scores_run(fi_scores *s, const fi_scores_args *a);

/* fi_scores_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_scores_destroy(fi_scores *s);

/*
 * The gated delta rule: linear attention that replaces what its state holds at
 * a key instead of adding to it.  For every row b, value head n, its key head
 * n / (Hv/Hk) and position t, with a = exp(log_decay[t][n]):
 *
 *     u[t] = beta[t][n] (v[t] - a S[t-1]^T k[t])
 *     S[t] = a S[t-1] + k[t] u[t]^T                (S is dk x dv)
 *     o[t] = scale * S[t]^T q[t]
 *
 * q, k, v and o are of io_dtype, log_decay and beta fp32; S is held, summed and
 * stored in fp32, and o is rounded to io_dtype once.  log_decay is <= 0, -inf for
 * a = 0 (what is left of a state over up to 64 positions may count as nothing below 2^-126 of it).  Keys of length one and beta in [0, 2] keep S bounded
 * (fi_rotary_run norms them); others are taken, and S grows as the formula
 * has it.  Calls run on the device that was current when the handle was made.
 * States, slots and rows out of the pool are as fi_lattn's; two rows of one call
 * must not share a slot unless the call holds.
 */
typedef struct fi_delta fi_delta;   /* opaque; owns its device memory */
typedef struct {
    int64_t B;                /* most rows of one call, >= 1 */
    int64_t L;                /* most positions of one fi_delta_prompt call, >= 1 */
    int64_t Hk;               /* query and key heads, >= 1 */
    int64_t Hv;               /* value heads, a multiple of Hk */
    int64_t dk, dv;           /* sizes of a key and of a value head, 1 .. 256 */
    float scale;              /* multiplies o; finite */
    fi_dtype io_dtype;        /* type of q, k, v and o */
    void *stream;             /* hipStream_t; NULL = the null stream */
} fi_delta_config;

typedef struct {
    int64_t B, L;             /* rows and positions of this call, within the config's */
    fi_view q, k, v;          /* [B][L][Hk][dk], [B][L][Hk][dk], [B][L][Hv][dv] */
    fi_view o;                /* [B][L][Hv][dv]; overlaps no input */
    fi_view log_decay, beta;  /* [B][L][Hv], fp32: the value of head n at position t of row b lies at p + b*row + t*pos + n*head */
    const int32_t *lens;      /* [B] on the device: row b has lens[b] positions (taken into [0, L]); NULL:
                                 all have L.  What lies past a row's end is not read as a number; o is zero there. */
    const int32_t *slots;     /* [B] on the device, or NULL */
    int64_t n_slots;          /* states in `state` (>= B where slots is NULL) */
    float *state;             /* read, and updated in place; aligned to 16 bytes; may be NULL in a fresh prompt */
    int32_t fresh;            /* nonzero: every row begins from S = 0, whatever its slot holds */
    int32_t hold;             /* nonzero: no state is changed (positions that may yet be taken back) */
} fi_delta_args;

/* fi_delta_create: allocates the workspace of the longest prompt: at most 437 MB for the systems of its chunks (64 positions;
 * fp32: 32), or 54 KB for each row and head where those are more than 8192; at most 101 MB for the states of segments;
 * and where all rows and heads have more than 32768 chunks, 4 dk dv bytes for each row and head.  Synchronous.
 * FI_ERR_INVALID for a NULL pointer, a size < 1, Hv not a multiple of Hk, an
 * infinite or NaN scale, an unknown dtype or sizes that overflow;
 * FI_ERR_UNSUPPORTED for dk or dv > 256, L > FI_MAX_L, B Hv > 2^20 or a device
 * that is not gfx950; FI_ERR_NOMEM / FI_ERR_HIP from the device. */
int fi_delta_create(const fi_delta_config *cfg, fi_delta **out);

/* fi_delta_prompt: L given positions of every row, from the row's state, which is
 * left after its last position.  B = 0 and L = 0 are allowed.  FI_ERR_INVALID
 * for a NULL pointer, sizes beyond the config's, fewer than B states without
 * slots, or a pointer that is not aligned to its element.  A NaN or infinity in
 * q, k, v or beta at t, or a NaN in log_decay, can make every output of its row
 * in the heads that read it, from up to 63 positions before t on, and their
 * states NaN or infinite; other rows and heads do not change. */
int fi_delta_prompt(fi_delta *s, const fi_delta_args *a);

/* fi_delta_step: one new position of every row in the recurrent form; L is 1,
 * lens NULL and state not NULL, also where fresh (else FI_ERR_INVALID).  Errors
 * as fi_delta_prompt. */
int fi_delta_step(fi_delta *s, const fi_delta_args *a);

/* fi_delta_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_delta_destroy(fi_delta *s);

/*
 * Queries and keys before a mixer: every head normed, and turned by its
 * position, in one pass.  For a head x[0 .. d) at position p:
 *
 *     FI_NORM_RMS: x[c] /= sqrt(sum_c x[c]^2 / d + eps)
 *     FI_NORM_L2:  x[c] /= sqrt(sum_c x[c]^2 + eps)
 *     x[c] *= w[c]                                     (where w is given)
 *     (x[a], x[b]) turned by p * inv_freq[i], i < rot/2:
 *         y[a] = x[a] cos - x[b] sin,  y[b] = x[b] cos + x[a] sin
 *
 * with (a, b) = (i, i + rot/2) or (2i, 2i + 1); elements from rot on are not
 * turned: what is not finite there reaches no other element but by the norm.  Everything is fp32, the sums of squares too (the angles are reduced in
 * 64 bits), rounded to io_dtype once.  Calls run on the device that was current when the handle was made.
 */
typedef enum { FI_NORM_NONE = 0, FI_NORM_RMS = 1, FI_NORM_L2 = 2 } fi_norm;
typedef enum { FI_PAIRS_HALVES = 0, FI_PAIRS_ADJACENT = 1 } fi_pairs;
typedef struct fi_rotary fi_rotary;   /* opaque; owns its device memory */
typedef struct {
    int64_t B, L;             /* most rows and positions of one call, >= 1 */
    int64_t Hq, Hk;           /* query heads, >= 1, and key heads, >= 0 */
    int64_t d;                /* size of a head, 1 .. 256 */
    int64_t rot;              /* elements of a head that are turned: even, 0 .. d */
    fi_norm norm;
    float eps;                /* finite, >= 0 */
    fi_pairs pairs;
    fi_dtype io_dtype;        /* type of the heads and of their weights */
    void *stream;             /* hipStream_t; NULL = the null stream */
} fi_rotary_config;
typedef struct {
    int64_t B, L;             /* rows and positions of this call, within the config's */
    fi_view q, k;             /* [B][L][Hq][d], [B][L][Hk][d]; k is ignored where Hk = 0 */
    fi_view qo, ko;           /* the results; each may be its input (the same pointer and strides), else overlaps no input */
    const void *wq, *wk;      /* [d] weights of the query (key) heads, or NULL */
    const int32_t *first;     /* [B] on the device: position t of row b stands at first[b] + t; or NULL: at t */
    const int32_t *positions; /* [B][L] on the device: where each position stands; or NULL.  Not with first. */
} fi_rotary_args;

/* fi_rotary_create: copies inv_freq[rot/2] (device, fp32, finite; NULL where rot
 * is 0).  Synchronous.  FI_ERR_INVALID for a NULL pointer, a size out of range, an odd
 * rot, eps negative or not finite, an unknown norm, pairs or dtype, an inv_freq that
 * is not finite or sizes that overflow; FI_ERR_UNSUPPORTED for d > 256 or a device that
 * is not gfx950; FI_ERR_NOMEM / FI_ERR_HIP from the device. */
int fi_rotary_create(const fi_rotary_config *cfg, const float *inv_freq, fi_rotary **out);

/* fi_rotary_run: B = 0 and L = 0 are allowed.  FI_ERR_INVALID for a NULL pointer,
 * sizes beyond the config's, a pointer that is not aligned to its element, or
 * first and positions both given. */
int fi_rotary_run(fi_rotary *s, const fi_rotary_args *a);

/* fi_rotary_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_rotary_destroy(fi_rotary *s);

/*
 * Drafted tokens against the target's probabilities, from given random numbers, so
 * that what comes out is distributed as the target's own tokens.  Row b
 * has lens[b] = n drafts x_0 .. x_{n-1}, the target's logits at each and behind the last,
 * p_i = softmax(scale z_i), and the logits that the drafts were drawn by,
 * q_i = softmax(draft_scale y_i) (without them the drafts are certain: q_i(x_i) = 1).
 *
 *     kept = the first i with u[i] q_i(x_i) >= p_i(x_i), n where there is none
 *     w = max(p_kept - q_kept, 0), and p_n where kept = n
 *     out = x_0 .. x_{kept-1}, then the first token j with w_j > 0 and
 *           w_0 + .. + w_j > r (w_0 + .. + w_{V-1}) (the last with w_j > 0 where there is none),
 *           then -1
 *     logprob = log p_i(out[i]), 0 behind the last
 *
 * all held in 64 bits (probabilities down to 2^-900 of the largest to 2^-38 of themselves; below 2^-1020 of it they
 * may count as none).  Where w is zero everywhere (a draft that neither allows), the token is
 * drawn from p_kept.  A logit of -inf is a token that is ruled out.  A draft
 * outside [0, V) is not kept.  Logits with a NaN or +inf, or without any token left, are no
 * distribution: a target's keep no draft, and out there is -1, logprob NaN; a draft's do not keep it
 * either, and the token is drawn from p_kept.  Calls run on the device that was current when the
 * handle was made.
 */
typedef struct fi_verify fi_verify;   /* opaque; owns its device memory */
#define FI_VERIFY_MAX_DRAFTS 63
typedef struct {
    int64_t B;                /* most rows of one call, >= 1 */
    int64_t N;                /* most drafts of a row, 0 .. FI_VERIFY_MAX_DRAFTS */
    int64_t V;                /* tokens of the vocabulary, 1 .. 2^31 - 1 */
    fi_dtype io_dtype;        /* type of the logits */
    float scale, draft_scale; /* finite, > 0 */
    void *stream;             /* hipStream_t; NULL = the null stream */
} fi_verify_config;
typedef struct {
    int64_t B, N;             /* rows and places for drafts of this call, within the config's */
    const void *target; int64_t target_row, target_ld;   /* [B][N+1][V]: rows target_row, positions target_ld elements apart, */
    const void *draft; int64_t draft_row, draft_ld;      /* [B][N][V]; any strides >= 0; draft may be NULL */
    const int64_t *tokens;    /* [B][N] drafts */
    const int32_t *lens;      /* [B] drafts of each row (taken into [0, N]), or NULL: all have N */
    const float *u;           /* [B][N] random numbers in [0, 1) for the drafts */
    const float *r;           /* [B] random numbers in [0, 1) for the token after them */
    int64_t *out;             /* [B][N+1] */
    int32_t *kept;            /* [B] */
    float *logprob;           /* [B][N+1], or NULL */
} fi_verify_args;

/* fi_verify_create: allocates the workspace.  FI_ERR_INVALID for a NULL pointer, a
 * size or scale out of range or an unknown dtype; FI_ERR_UNSUPPORTED for B (2 N + 1) > 2^22 or
 * when the device is not gfx950; FI_ERR_NOMEM / FI_ERR_HIP from the device. */
int fi_verify_create(const fi_verify_config *cfg, fi_verify **out);

/* fi_verify_run: FI_ERR_INVALID for a NULL handle, args, target, r, out or kept, for NULL
 * tokens or u where N > 0, sizes beyond the config's, a negative stride, or a
 * pointer not aligned to its element. */
int fi_verify_run(fi_verify *s, const fi_verify_args *a);

/* fi_verify_destroy: synchronise the stream and free everything; NULL is a no-op. */
void fi_verify_destroy(fi_verify *s);

#ifdef __cplusplus
}
#endif
#endif /* FI_H_ */
