// kda_selective_api.hip -- the C ABI of the short convolution and the selective
// scan (declared in include/kda_selective.h).  As in kda_api.hip every entry
// point validates its arguments synchronously, before any launch, and launches
// on the caller's stream; nothing here allocates or keeps state.
#include <stdint.h>

#include "kda_checks.hpp"
#include "kda_selective.h"
#include "kda_selective_internal.hpp"

using namespace kda;

namespace {

bool ok_io(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }

// a * b, or INT64_MAX where that does not fit (a, b >= 0)
int64_t mul_sat(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}

// What both operators ask of their rows.  Token indices and a row's bytes are
// 32-bit in the kernels, elements 64-bit.
kda_status check_rows(int64_t batch, int64_t seqlen, int64_t width, int64_t n_seq, kda_dtype io) {
    if (batch < 0 || seqlen < 0 || width <= 0 || n_seq < -1 || !ok_io(io)) return KDA_ERR_INVALID_ARGUMENT;
    if (n_seq >= 0 && batch != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (seqlen > (1 << 30) || width > (1 << 28) || batch > (1 << 24) || n_seq > (1 << 24) ||
        mul_sat(mul_sat(batch, seqlen), width) > ((int64_t)1 << 40))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// ---- short convolution ------------------------------------------------------

ShortConvArgs conv_args(const kda_short_conv_problem* p) {
    ShortConvArgs a = {};
    a.B = p->batch; a.T = p->seqlen; a.D = p->width; a.n_seq = p->n_seq >= 0 ? p->n_seq : p->batch;
    a.taps = p->taps; a.silu = p->silu != 0;
    return a;
}

kda_status check_taps(int32_t taps, int32_t silu) {
    if (taps < 1 || (silu != 0 && silu != 1)) return KDA_ERR_INVALID_ARGUMENT;
    return taps < 2 || taps > 4 ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

kda_status check_conv(const kda_short_conv_problem* p) {
    if (!p) return KDA_ERR_INVALID_ARGUMENT;
    kda_status st = check_rows(p->batch, p->seqlen, p->width, p->n_seq, p->io_dtype);
    if (st != KDA_OK) return st;
    if ((st = check_taps(p->taps, p->silu)) != KDA_OK) return st;
    return short_conv_fits(conv_args(p), p->io_dtype == KDA_BF16) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

bool ok_offsets(int64_t n_seq, const int32_t* cu) { return n_seq >= 0 ? ok_elem(cu, true, 4) : cu == nullptr; }

// ---- selective scan ---------------------------------------------------------

SelectiveArgs scan_args(const kda_selective_scan_problem* p) {
    SelectiveArgs a = {};
    a.B = p->batch; a.T = p->seqlen; a.D = p->width; a.n_seq = p->n_seq >= 0 ? p->n_seq : p->batch;
    a.states = p->states;
    return a;
}

// The workspaces of a packed batch are larger; sizes go by whether it is one.
const int32_t kPacked = 0;

kda_status check_states(int32_t states) {
    if (states < 1) return KDA_ERR_INVALID_ARGUMENT;
    return states == 8 || states == 16 || states == 32 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status check_scan(const kda_selective_scan_problem* p) {
    if (!p) return KDA_ERR_INVALID_ARGUMENT;
    kda_status st = check_rows(p->batch, p->seqlen, p->width, p->n_seq, p->io_dtype);
    if (st != KDA_OK) return st;
    if ((st = check_states(p->states)) != KDA_OK) return st;
    if (mul_sat(mul_sat(p->n_seq >= 0 ? p->n_seq : p->batch, p->width), p->states) > ((int64_t)1 << 40)) return KDA_ERR_UNSUPPORTED;
    return selective_scan_fits(scan_args(p)) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

size_t scan_bytes(const kda_selective_scan_problem* p, bool backward) {
    SelectiveArgs a = scan_args(p);
    if (p->n_seq >= 0) a.cu_seqlens = &kPacked;      // not read
    return selective_scan_workspace_bytes(a, backward);
}

kda_status check_inputs(const kda_selective_scan_problem* p, const kda_selective_scan_inputs* in) {
    if (!in) return KDA_ERR_INVALID_ARGUMENT;
    const bool any = p->batch > 0 && p->seqlen > 0;
    if (!ok_ptr(in->x, any) || !ok_ptr(in->dt, any) || !ok_ptr(in->A, true) || !ok_ptr(in->B, any) || !ok_ptr(in->C, any) ||
        !ok_opt_ptr(in->skip) || !ok_opt_ptr(in->z) || !ok_opt_ptr(in->dt_bias) || !ok_opt_ptr(in->state_in) ||
        !ok_offsets(p->n_seq, in->cu_seqlens))
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

void set_inputs(SelectiveArgs& a, const kda_selective_scan_inputs* in) {
    a.x = in->x; a.dt = in->dt; a.A = in->A; a.Bm = in->B; a.Cm = in->C; a.skip = in->skip; a.z = in->z;
    a.dt_bias = in->dt_bias; a.state_in = in->state_in; a.cu_seqlens = in->cu_seqlens;
}

kda_status scan_forward(const kda_selective_scan_problem* p, const kda_selective_scan_inputs* in, void* out,
                        float* state_out, void* workspace, size_t workspace_bytes, bool keep, void* stream) {
    kda_status st = check_scan(p);
    if (st != KDA_OK) return st;
    if ((st = check_inputs(p, in)) != KDA_OK) return st;
    const bool any = p->batch > 0 && p->seqlen > 0;
    const size_t need = scan_bytes(p, keep);
    if (!ok_ptr(out, any) || !ok_opt_ptr(state_out) || !ok_ptr(workspace, need > 0)) return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
    SelectiveArgs a = scan_args(p);
    if (a.n_seq == 0 || (!any && !state_out)) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    set_inputs(a, in);
    a.out = out; a.state_out = state_out; a.keep = keep; a.ws = static_cast<char*>(workspace);
    return hip_status(launch_selective_scan(p->io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

}  // namespace

extern "C" {

kda_status kda_short_conv_prefill(const kda_short_conv_problem* p, const void* x, const float* weight,
                                  const float* bias, const void* state_in, const int32_t* cu_seqlens, void* out,
                                  void* state_out, void* stream) {
    kda_status st = check_conv(p);
    if (st != KDA_OK) return st;
    const bool any = p->batch > 0 && p->seqlen > 0;
    if (!ok_ptr(x, any) || !ok_ptr(weight, true) || !ok_opt_ptr(bias) || !ok_opt_ptr(state_in) ||
        !ok_offsets(p->n_seq, cu_seqlens) || !ok_ptr(out, any) || !ok_opt_ptr(state_out))
        return KDA_ERR_INVALID_ARGUMENT;
    if (any && out == x) return KDA_ERR_INVALID_ARGUMENT;       // tiles read the inputs before them
    ShortConvArgs a = conv_args(p);
    if (a.n_seq == 0 || (!any && !state_out)) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    a.cu_seqlens = cu_seqlens; a.x = x; a.weight = weight; a.bias = bias; a.state_in = state_in; a.out = out;
    a.state_out = state_out;
    return hip_status(launch_short_conv(p->io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

size_t kda_short_conv_backward_workspace_size(const kda_short_conv_problem* p) {
    if (check_conv(p) != KDA_OK) return 0;
    return short_conv_backward_workspace_bytes(conv_args(p), p->io_dtype == KDA_BF16);
}

kda_status kda_short_conv_backward(const kda_short_conv_problem* p, const void* x, const float* weight,
                                   const float* bias, const void* state_in, const int32_t* cu_seqlens,
                                   const void* d_out, const void* d_state, void* dx, float* dweight, float* dbias,
                                   void* d_state_in, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st = check_conv(p);
    if (st != KDA_OK) return st;
    const bool any = p->batch > 0 && p->seqlen > 0;
    const size_t need = kda_short_conv_backward_workspace_size(p);
    if (!ok_ptr(x, any) || !ok_ptr(weight, true) || !ok_opt_ptr(bias) || !ok_opt_ptr(state_in) ||
        !ok_offsets(p->n_seq, cu_seqlens) || !ok_opt_ptr(d_out) || !ok_opt_ptr(d_state) || !ok_ptr(dx, any) ||
        !ok_ptr(dweight, true) || !ok_ptr(dbias, bias != nullptr) || !ok_opt_ptr(d_state_in) ||
        !ok_ptr(workspace, need > 0))
        return KDA_ERR_INVALID_ARGUMENT;
    if (any && (dx == x || (d_out && dx == d_out))) return KDA_ERR_INVALID_ARGUMENT;     // tiles read beyond their ends
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if ((st = device_ready()) != KDA_OK) return st;
    ShortConvArgs a = conv_args(p);
    a.cu_seqlens = cu_seqlens; a.x = x; a.weight = weight; a.bias = bias; a.state_in = state_in; a.d_out = d_out;
    a.d_state = d_state; a.dx = dx; a.dweight = dweight; a.dbias = bias ? dbias : nullptr; a.d_state_in = d_state_in;
    a.parts = static_cast<float*>(workspace);
    return hip_status(launch_short_conv_backward(p->io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

kda_status kda_short_conv_step(int64_t N, int64_t width, int32_t taps, int32_t silu, kda_dtype io_dtype, const void* x,
                               const float* weight, const float* bias, void* state, void* out, void* stream) {
    if (N < 0 || width <= 0 || !ok_io(io_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    kda_status st = check_taps(taps, silu);
    if (st != KDA_OK) return st;
    if (mul_sat(N, width) > UINT32_MAX - 255) return KDA_ERR_UNSUPPORTED;      // threads of a launch
    const bool any = N > 0;
    if (!ok_ptr(x, any) || !ok_ptr(weight, any) || !ok_opt_ptr(bias) || !ok_ptr(state, any) || !ok_ptr(out, any))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!any) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    ShortConvStepArgs a = {};
    a.N = N; a.D = width; a.taps = taps; a.silu = silu != 0; a.x = x; a.weight = weight; a.bias = bias; a.state = state;
    a.out = out;
    return hip_status(launch_short_conv_step(io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

size_t kda_selective_scan_workspace_size(const kda_selective_scan_problem* p) {
    return check_scan(p) == KDA_OK ? scan_bytes(p, false) : 0;
}

size_t kda_selective_scan_backward_workspace_size(const kda_selective_scan_problem* p) {
    return check_scan(p) == KDA_OK ? scan_bytes(p, true) : 0;
}

kda_status kda_selective_scan_prefill(const kda_selective_scan_problem* p, const kda_selective_scan_inputs* in,
                                      void* out, float* state_out, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    return scan_forward(p, in, out, state_out, workspace, workspace_bytes, false, stream);
}

kda_status kda_selective_scan_prefill_for_backward(const kda_selective_scan_problem* p,
                                                   const kda_selective_scan_inputs* in, void* out, float* state_out,
                                                   void* workspace, size_t workspace_bytes, void* stream) {
    return scan_forward(p, in, out, state_out, workspace, workspace_bytes, true, stream);
}

kda_status kda_selective_scan_backward(const kda_selective_scan_problem* p, const kda_selective_scan_inputs* in,
                                       const void* d_out, const float* d_state,
                                       const kda_selective_scan_gradients* to, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    kda_status st = check_scan(p);
    if (st != KDA_OK) return st;
    if ((st = check_inputs(p, in)) != KDA_OK) return st;
    if (!to) return KDA_ERR_INVALID_ARGUMENT;
    const bool any = p->batch > 0 && p->seqlen > 0;
    const size_t need = scan_bytes(p, true);
    if (!ok_opt_ptr(d_out) || !ok_opt_ptr(d_state) || !ok_ptr(to->dx, any) || !ok_ptr(to->ddt, any) ||
        !ok_ptr(to->dA, true) || !ok_ptr(to->dB, any) || !ok_ptr(to->dC, any) ||
        !ok_ptr(to->dskip, in->skip != nullptr) || !ok_ptr(to->dz, any && in->z != nullptr) ||
        !ok_ptr(to->ddt_bias, in->dt_bias != nullptr) || !ok_opt_ptr(to->d_state_in) || !ok_ptr(workspace, need > 0))
        return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if ((st = device_ready()) != KDA_OK) return st;
    SelectiveArgs a = scan_args(p);
    set_inputs(a, in);
    a.d_out = d_out; a.d_state = d_state; a.dx = to->dx; a.ddt = to->ddt; a.dA = to->dA; a.dB = to->dB; a.dC = to->dC;
    a.dskip = in->skip ? to->dskip : nullptr; a.dz = to->dz; a.ddt_bias = in->dt_bias ? to->ddt_bias : nullptr;
    a.d_state_in = to->d_state_in; a.ws = static_cast<char*>(workspace);
    return hip_status(launch_selective_scan_backward(p->io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

kda_status kda_selective_scan_step(int64_t N, int64_t width, int32_t states, kda_dtype io_dtype, const void* x,
                                   const void* dt, const float* A, const void* B, const void* C, const float* skip,
                                   const void* z, const float* dt_bias, float* state, void* out, void* stream) {
    if (N < 0 || width <= 0 || !ok_io(io_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    kda_status st = check_states(states);
    if (st != KDA_OK) return st;
    if (mul_sat(mul_sat(N, width), states / 4) > UINT32_MAX - 255) return KDA_ERR_UNSUPPORTED;      // threads of a launch
    const bool any = N > 0;
    if (!ok_ptr(x, any) || !ok_ptr(dt, any) || !ok_ptr(A, any) || !ok_ptr(B, any) || !ok_ptr(C, any) || !ok_opt_ptr(skip) ||
        !ok_opt_ptr(z) || !ok_opt_ptr(dt_bias) || !ok_ptr(state, any) || !ok_ptr(out, any))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!any) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    SelectiveArgs a = {};
    a.B = N; a.T = 1; a.D = width; a.n_seq = N; a.states = states; a.x = x; a.dt = dt; a.A = A; a.Bm = B; a.Cm = C; a.skip = skip;
    a.z = z; a.dt_bias = dt_bias; a.state_out = state; a.out = out;
    return hip_status(launch_selective_scan_step(io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

}  // extern "C"
