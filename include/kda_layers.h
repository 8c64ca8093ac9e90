/*
 * kda_layers.h -- C ABI of the operators around the KDA chunk recurrence in a layer of a language
 * model: the short causal convolution in front of it, the selective state space scan (the
 * diagonal-state recurrence that takes its place in other layers), the norm of its output per
 * group of channels, and the single-token forms with which a model is served.
 *
 * Conventions are those of kda.h: DEVICE pointers owned by the caller, work enqueued on `stream`
 * of the current HIP device with no allocation, no synchronisation and no state kept between
 * calls; arguments checked before any HIP call (KDA_EINVAL / KDA_EUNSUPPORTED with a message
 * from kda_last_error()); sums in fp32 in a fixed order, so results are the same from run to run.
 * Every call may be captured into a HIP graph; sizes and cuts are those of the capture, and the device
 * copy of the cuts still holds them at every replay.
 *
 * Token axis: dense batches are [B, T, ...]; packed sequences have B = 1, T tokens in all and
 * cu_seqlens (device and host copies with the same values) with N sequences, empty ones allowed.
 *
 * Outputs and the workspace overlap neither each other nor an input; `state` of a token step is the
 * only argument that is read and written.
 *
 * Rows: tensors are contiguous, except that an input named with a *_row field may be a column
 * slice of a wider contiguous matrix: its element (token i, column c) is at i * row + c, tokens
 * counted over the whole batch. A row of 0 means the tensor's own width.
 *
 * Element types: inputs and outputs marked dtype are fp32 or bf16; the rest is fp32. All
 * arithmetic is fp32; outputs are rounded once, to nearest even.
 */
#ifndef KDA_LAYERS_H
#define KDA_LAYERS_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1, KDA_ACT_SIGMOID = 2 } kda_act;

/* ---------------------------------------------------------------------------------------------
 * Short causal convolution, one filter per channel:
 *   u_t = bias + sum_{j < W} weight[:, j] x_{t - (W-1) + j},   y_t = act(u_t),
 * where the W - 1 rows before a sequence's first token are h0 (zero without one).
 */
typedef struct {
    int32_t B, T;          /* tokens as above; T >= 0                                            */
    int32_t D;             /* channels                                                           */
    int32_t W;             /* taps: 2, 3 or 4                                                    */
    int32_t N;             /* sequences: B when dense                                            */
    const int32_t* cu_seqlens_dev;
    const int32_t* cu_seqlens_host;
    int64_t x_row;         /* row of x                                                           */
    int32_t act;           /* KDA_ACT_NONE or KDA_ACT_SILU                                       */
    int32_t dtype;         /* kda_dtype                                                          */
} kda_conv_dims;

/*
 *   x [B,T,D] dtype, weight [D,W] fp32, bias [D] fp32 or NULL, h0 [N,W-1,D] dtype or NULL
 *   y [B,T,D] dtype; final_state [N,W-1,D] dtype (the last W - 1 rows of [h0 | x]) or NULL
 */
kda_status kda_short_conv_fwd(const kda_conv_dims* dims, const void* x, const float* weight, const float* bias,
                              const void* h0, void* y, void* final_state, void* stream);

/* Workspace of the backward; 0 if dims are invalid. 256-byte aligned, any contents. */
size_t kda_short_conv_bwd_workspace_bytes(const kda_conv_dims* dims);

/*
 * Gradients of sum<dy, y> + <dfinal, final_state> (dfinal [N,W-1,D] dtype or NULL = zero):
 *   dx [B,T,D] dtype, dweight [D,W] fp32, dbias [D] fp32 or NULL, dh0 [N,W-1,D] dtype or NULL
 */
kda_status kda_short_conv_bwd(const kda_conv_dims* dims, const void* x, const float* weight, const float* bias,
                              const void* h0, const void* dy, const void* dfinal, void* dx, float* dweight,
                              float* dbias, void* dh0, void* workspace, size_t ws_bytes, void* stream);

/*
 * One token of each of dims->B sequences (T = 1, no cu_seqlens, N = B). state [S,W-1,D] dtype is
 * updated in place: row slots[b] (int32 [B], NULL: row b) drops its oldest input and takes x.
 * A negative slot marks a padding row: no state is touched and its y is zero. A slot >= S, or
 * one that an earlier row of the call has too, is refused: no state is touched, its y is NaN.
 */
kda_status kda_short_conv_step(const kda_conv_dims* dims, const void* x, const float* weight, const float* bias,
                               const int32_t* slots, int32_t S, void* state, void* y, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Selective state space scan. With dt_t = raw_t + dt_bias (softplus of it where dims->softplus):
 *   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = <C_t, h_t> + skip x_t,   y_t *= silu(z_t),
 * per channel d with NS states; B and C are shared by the D / G channels of a group. Where NS is 8,
 * 16, 32 or 64, the fp32 arrays with a last dimension NS must be 16-byte aligned.
 */
#define KDA_SCAN_CHUNK 16 /* tokens between two saved states */

typedef struct {
    int32_t B, T;
    int32_t D;             /* channels                                                           */
    int32_t NS;            /* states per channel, 1 .. 64                                        */
    int32_t G;             /* groups of B and C; D % G == 0                                      */
    int32_t N;             /* sequences                                                          */
    const int32_t* cu_seqlens_dev;
    const int32_t* cu_seqlens_host;
    int64_t x_row, dt_row, z_row, b_row, c_row;
    int32_t softplus;      /* 0 or 1                                                             */
    int32_t dtype;         /* of x, raw dt, z, B, C, dy and y, dx, ddt, dz, dB, dC               */
} kda_sscan_dims;

/* Chunks that the saved states cover: sum over sequences of ceil(len / KDA_SCAN_CHUNK); -1 if
 * dims are invalid. */
int64_t kda_sscan_num_chunks(const kda_sscan_dims* dims);
size_t kda_sscan_fwd_workspace_bytes(const kda_sscan_dims* dims);
size_t kda_sscan_bwd_workspace_bytes(const kda_sscan_dims* dims);

/*
 *   x, dt [B,T,D] dtype; A [D,NS] fp32; Bm, Cm [B,T,G,NS] dtype; skip [D] fp32 or NULL;
 *   z [B,T,D] dtype or NULL; dt_bias [D] fp32 or NULL; h0 [N,D,NS] fp32 or NULL
 *   y [B,T,D] dtype; final_state [N,D,NS] fp32 or NULL (h0 for an empty sequence);
 *   states [chunks,D,NS] fp32 or NULL: the state entering each chunk, for the backward
 */
kda_status kda_sscan_fwd(const kda_sscan_dims* dims, const void* x, const void* dt, const float* A, const void* Bm,
                         const void* Cm, const float* skip, const void* z, const float* dt_bias, const float* h0,
                         void* y, float* final_state, float* states, void* workspace, size_t ws_bytes,
                         void* stream);

/*
 * Gradients of sum<dy, y> + <dfinal, final_state> (dfinal [N,D,NS] fp32 or NULL = zero), from the
 * states that kda_sscan_fwd saved for the same arguments:
 *   dx, ddt [B,T,D] dtype (ddt: of the raw dt), dA [D,NS] fp32, dB, dC [B,T,G,NS] dtype;
 *   dskip [D] (needs skip), dz [B,T,D] dtype (needs z), ddt_bias [D], dh0 [N,D,NS] fp32: each may be
 *   NULL
 */
kda_status kda_sscan_bwd(const kda_sscan_dims* dims, const void* x, const void* dt, const float* A, const void* Bm,
                         const void* Cm, const float* skip, const void* z, const float* dt_bias,
                         const float* states, const void* dy, const float* dfinal, void* dx, void* ddt, float* dA,
                         void* dB, void* dC, float* dskip, void* dz, float* ddt_bias, float* dh0, void* workspace,
                         size_t ws_bytes, void* stream);

/* One token of each of dims->B sequences; state [S,D,NS] fp32 in place, slots as above. */
kda_status kda_sscan_step(const kda_sscan_dims* dims, const void* x, const void* dt, const float* A, const void* Bm,
                          const void* Cm, const float* skip, const void* z, const float* dt_bias,
                          const int32_t* slots, int32_t S, float* state, void* y, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Norm over each group of C channels of a row, channels last, with an activation:
 *   n = (x - mean) rstd (center) or x / sqrt(mean(x^2) + eps),   u = n weight + bias,
 *   y = act(u), or u act(gate) with a gate.
 * Statistics are per row (token), so that a token's output depends on no other token.
 */
typedef struct {
    int64_t R;             /* rows                                                               */
    int32_t G, C;          /* groups of a row; channels of a group, 1 .. 8192                    */
    int32_t center;        /* 1: subtract the mean. 0: root mean square only                     */
    int32_t act;           /* kda_act                                                            */
    int32_t shared;        /* 1: weight and bias are [C], one for all groups. 0: [G*C]           */
    float eps;             /* > 0                                                                */
    int64_t x_row, gate_row;
    int32_t dtype;
} kda_norm_dims;

/* x [R,G*C] dtype, weight and bias fp32 (each may be NULL: 1 and 0), gate [R,G*C] dtype or NULL;
 * y [R,G*C] dtype */
kda_status kda_group_norm_fwd(const kda_norm_dims* dims, const void* x, const float* weight, const float* bias,
                              const void* gate, void* y, void* stream);
size_t kda_group_norm_bwd_workspace_bytes(const kda_norm_dims* dims);
/* dx [R,G*C] dtype; dweight, dbias as weight and bias (NULL: not written); dgate [R,G*C] dtype
 * (with a gate) */
kda_status kda_group_norm_bwd(const kda_norm_dims* dims, const void* x, const float* weight, const float* bias,
                              const void* gate, const void* dy, void* dx, float* dweight, float* dbias, void* dgate,
                              void* workspace, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------------------------
 * One token of KDA for each of dims->B sequences (dims->T = 1, N = B, no cu_seqlens; C is not
 * read; K and V up to 256):
 *   S' = Diag(e^g) S,  u = beta (v - S'^T k),  S <- S' + k u^T,  o = scale S^T q.
 *   q, k [B,H,K] dtype, v [B,HV,V] dtype, g [B,HV,K] fp32, beta [B,HV] fp32 (logits where
 *   dims->beta_logits), state [S,HV,K,V] fp32 in place (kda_fwd_states' final_state is one),
 *   slots as above, o [B,HV,V] dtype
 */
kda_status kda_step(const kda_dims* dims, const void* q, const void* k, const void* v, const float* g,
                    const float* beta, const int32_t* slots, int32_t S, float* state, void* o, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LAYERS_H */
