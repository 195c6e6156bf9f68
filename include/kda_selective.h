/*
 * kda_selective.h -- C ABI of two more operators of libkda.so that stand beside
 * KDA in a hybrid stack, with their gradients and their single-token forms: the
 * short causal convolution that the inputs of a recurrent mixer pass, and a
 * selective state space, a linear recurrence whose steps, writes and reads
 * depend on the token.
 *
 * The conventions are those of kda.h: device pointers, C-contiguous and
 * 16-byte aligned (int32 arrays need 4-byte alignment), an asynchronous call on
 * `stream`, memory owned by the caller, nothing launched after a refused
 * argument, nothing on the stream but kernel launches (so every call can be
 * captured into a HIP graph and replayed).  Outputs may not overlap each other
 * or the inputs except where a call says so, and a workspace serves one call at
 * a time.  A launch holds fewer than 2^32 threads; a problem that takes more is
 * KDA_ERR_UNSUPPORTED.  Results do not depend on timing: sums over tokens and
 * channels are taken in a fixed order.
 *
 * Packed batches are those of kda_varlen_prepare: batch == 1 and cu_seqlens of
 * n_seq + 1 offsets, which must not decrease (they are bounded, so that no
 * value makes an access leave the arrays; others give unspecified rows).  Tokens
 * of no sequence are not written, and add nothing to gradients of parameters.
 * An empty sequence passes its state, and its state's gradient, through.
 *
 * Sources: zuoshipin.com/article/18261 section 2 (recurrent memory with
 * channel-wise retention in a hybrid stack); devpress.csdn.net K3 article
 * section 14 (states kept at the boundaries of shared prefixes).  The pages
 * print no formula; those below define the calls.
 */
#ifndef KDA_SELECTIVE_H_
#define KDA_SELECTIVE_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- a short causal convolution -----------------------------------------------
 * Each channel is convolved with `taps` weights of its own:
 *   y_t   = bias + sum_(j < taps) weight[j] x_(t - taps + 1 + j)
 *   out_t = y_t sigmoid(y_t)        (silu; else out_t = y_t)
 * where the inputs before a sequence's first token are its state, the last
 * taps - 1 inputs seen so far (oldest first; zeros where no state is given).
 * Sums are fp32. */
typedef struct {
    int64_t batch;          /* rows; 1 for a packed batch                        */
    int64_t seqlen;         /* tokens of a row                                   */
    int64_t width;          /* channels, >= 1                                    */
    int64_t n_seq;          /* sequences of a packed batch; -1: not packed       */
    int32_t taps;           /* 2, 3 or 4                                         */
    int32_t silu;           /* 1: SiLU on the result, 0: none                    */
    kda_dtype io_dtype;     /* dtype of x, out, the states and their gradients   */
} kda_short_conv_problem;

/*   x, out: [batch, seqlen, width] io_dtype; weight: [width, taps] fp32; bias:
 *   [width] fp32 or NULL; state_in, state_out: [batch or n_seq, taps - 1, width]
 *   io_dtype, either may be NULL and they may be one array. */
kda_status kda_short_conv_prefill(const kda_short_conv_problem* p, const void* x, const float* weight,
                                  const float* bias, const void* state_in, const int32_t* cu_seqlens, void* out,
                                  void* state_out, void* stream);

/* Bytes of scratch for the call below; 0 where none is needed or p is invalid. */
size_t kda_short_conv_backward_workspace_size(const kda_short_conv_problem* p);

/* Gradients of <d_out, out> + <d_state, final states>, from the inputs alone.
 * d_out, d_state may be NULL (zero).  dx io_dtype, dweight fp32, dbias fp32
 * (written where bias is given, and may be NULL otherwise), d_state_in io_dtype
 * or NULL; all are overwritten. */
kda_status kda_short_conv_backward(const kda_short_conv_problem* p, const void* x, const float* weight,
                                   const float* bias, const void* state_in, const int32_t* cu_seqlens,
                                   const void* d_out, const void* d_state, void* dx, float* dweight, float* dbias,
                                   void* d_state_in, void* workspace, size_t workspace_bytes, void* stream);

/* One token of each of N sequences: x, out [N, width], state [N, taps - 1,
 * width] in place. */
kda_status kda_short_conv_step(int64_t N, int64_t width, int32_t taps, int32_t silu, kda_dtype io_dtype, const void* x,
                               const float* weight, const float* bias, void* state, void* out, void* stream);

/* ---- a selective state space ----------------------------------------------------
 * Per batch row and channel d, `states` states h_n (fp32), and for token t
 *   delta = softplus(dt_t + dt_bias)
 *   h_n   <- exp(delta A[d, n]) h_n + delta x_t B_t[n]
 *   y_t   = sum_n C_t[n] h_n + skip x_t
 *   out_t = y_t z_t sigmoid(z_t)        (z NULL: out_t = y_t)
 * B_t and C_t are shared by a row's channels.  A is finite and at most 0 (not
 * checked): a state then fades.  States, sums and the gradients' sums are fp32. */
typedef struct {
    int64_t batch;          /* rows; 1 for a packed batch                        */
    int64_t seqlen;         /* tokens of a row                                   */
    int64_t width;          /* channels, >= 1                                    */
    int64_t n_seq;          /* sequences of a packed batch; -1: not packed       */
    int32_t states;         /* states of a channel: 8, 16 or 32                  */
    kda_dtype io_dtype;     /* dtype of x, dt, B, C, z, out and their gradients  */
} kda_selective_scan_problem;

/* The inputs of a call.  x, dt, z: [batch, seqlen, width] io_dtype, z may be
 * NULL; A: [width, states] fp32; B, C: [batch, seqlen, states] io_dtype; skip,
 * dt_bias: [width] fp32 or NULL (zero); state_in: [batch or n_seq, width, states]
 * fp32 or NULL; cu_seqlens: NULL where n_seq is -1. */
typedef struct {
    const void* x;
    const void* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* skip;
    const void* z;
    const float* dt_bias;
    const float* state_in;
    const int32_t* cu_seqlens;
} kda_selective_scan_inputs;

/* Bytes of scratch for the calls below; 0 where none is needed or p is invalid. */
size_t kda_selective_scan_workspace_size(const kda_selective_scan_problem* p);
size_t kda_selective_scan_backward_workspace_size(const kda_selective_scan_problem* p);

/* out: as x; state_out: as state_in, may be NULL or state_in itself. */
kda_status kda_selective_scan_prefill(const kda_selective_scan_problem* p, const kda_selective_scan_inputs* in,
                                      void* out, float* state_out, void* workspace, size_t workspace_bytes,
                                      void* stream);

/* The same, leaving in a backward workspace the states that
 * kda_selective_scan_backward continues from. */
kda_status kda_selective_scan_prefill_for_backward(const kda_selective_scan_problem* p,
                                                   const kda_selective_scan_inputs* in, void* out, float* state_out,
                                                   void* workspace, size_t workspace_bytes, void* stream);

/* Where the gradients go: of the type and shape of what they belong to, all
 * overwritten.  dz, dskip and ddt_bias are written where z, skip and dt_bias are
 * given and may be NULL otherwise; d_state_in may be NULL. */
typedef struct {
    void* dx;
    void* ddt;
    float* dA;
    void* dB;
    void* dC;
    float* dskip;
    void* dz;
    float* ddt_bias;
    float* d_state_in;
} kda_selective_scan_gradients;

/* Gradients of <d_out, out> + <d_state, final states>, from the same inputs and
 * the workspace that the call above filled with them (state_in unchanged too:
 * not the array that state_out went to).  d_out, d_state may be NULL (zero).
 * The workspace can serve further backward calls. */
kda_status kda_selective_scan_backward(const kda_selective_scan_problem* p, const kda_selective_scan_inputs* in,
                                       const void* d_out, const float* d_state,
                                       const kda_selective_scan_gradients* to, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* One token of each of N sequences: x, dt, z, out [N, width], B, C [N, states],
 * state [N, width, states] fp32 in place. */
kda_status kda_selective_scan_step(int64_t N, int64_t width, int32_t states, kda_dtype io_dtype, const void* x,
                                   const void* dt, const float* A, const void* B, const void* C, const float* skip,
                                   const void* z, const float* dt_bias, float* state, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_SELECTIVE_H_ */
