// kda_recurrence.hip -- a gated linear recurrence per channel, its gradients
// and its single-token step.
//
//   lambda = max(log_alpha, floor),  h_t = e^lambda_t h_(t-1) + x_t,
//   out_t = h_t sigmoid(g_t)
// and in reverse, with dh_t the gradient of h_t:
//   dh_t = d_out_t sigmoid(g_t) + e^lambda_(t+1) dh_(t+1)   (d_state at the end)
//   dx_t = dh_t,  dlog_alpha_t = dh_t e^lambda_t h_(t-1)    (0 where the floor binds)
//   dg_t = d_out_t h_t sigmoid'(g_t),  d_state_in = e^lambda_0 dh_0
//
// A channel that remembers n tokens multiplies about n factors next to 1, so
// where |lambda| <= 1/4 a step is taken as h + (expm1(lambda) h + x): rounding
// e^lambda itself would cost half a step of fp32 per token, always the same
// way for a constant lambda.  Faster decays take e^lambda h + x, which leaves
// nothing of a large h that is forgotten.
#include "kda_common.hpp"
#include "kda_hybrid_internal.hpp"

namespace kda {

namespace {

constexpr int kTile = 64;     // tokens between kept states

// One token's decay, of lambda = max(log_alpha, floor): `c` is expm1(lambda)
// where `slow` and e^lambda elsewhere.  expm1 is the Taylor series to the 8th
// power (the rest is below 2^-31 of the value), e^lambda the hardware exp2.
struct Decay {
    float c;
    bool slow;
    __device__ __forceinline__ explicit Decay(float x) {
        float p = 1.f / 40320.f;
        p = fmaf(p, x, 1.f / 5040.f);
        p = fmaf(p, x, 1.f / 720.f);
        p = fmaf(p, x, 1.f / 120.f);
        p = fmaf(p, x, 1.f / 24.f);
        p = fmaf(p, x, 1.f / 6.f);
        p = fmaf(p, x, 0.5f);
        p = fmaf(p * x, x, x);
        slow = fabsf(x) <= 0.25f;
        c = slow ? p : __builtin_amdgcn_exp2f(1.4426950408889634f * x);
    }
    // e^lambda h, and e^lambda h + x
    __device__ __forceinline__ float times(float h) const { return fmaf(c, h, slow ? h : 0.f); }
    __device__ __forceinline__ float step(float h, float x) const { return fmaf(c, h, x) + (slow ? h : 0.f); }
};

struct Span {
    int64_t row, first, end;   // tokens [first, end) of batch row `row`; states at index blockIdx.y
};
__device__ __forceinline__ Span span_of(const RecurrenceArgs& a) {
    Span s;
    if (a.cu_seqlens) {
        s.row = 0;
        seq_bounds(a.cu_seqlens, blockIdx.y, a.T, s.first, s.end);
    } else {
        s.row = blockIdx.y; s.first = 0; s.end = a.T;
    }
    return s;
}

__device__ __forceinline__ int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }

template <typename E>
__global__ __launch_bounds__(64) void kda_recurrence_kernel(RecurrenceArgs a) {
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (c >= a.D) return;
    const Span sp = span_of(a);
    float h = a.state_in ? a.state_in[(int64_t)blockIdx.y * a.D + c] : 0.f;
    float* keep = reinterpret_cast<float*>(a.ws);
    for (int64_t t = sp.first; t < sp.end; ++t) {
        const int64_t i = (sp.row * a.T + t) * a.D + c;
        if (a.keep && t % kTile == 0) keep[(sp.row * tiles_of(a.T) + t / kTile) * a.D + c] = h;
        h = Decay(fmaxf(a.log_alpha[i], a.floor_)).step(h, to_f32(reinterpret_cast<const E*>(a.x)[i]));
        const float s = a.g ? sigmoidf_(to_f32(reinterpret_cast<const E*>(a.g)[i])) : 1.f;
        reinterpret_cast<E*>(a.out)[i] = from_f32<E>(h * s);
    }
    if (a.state_out) a.state_out[(int64_t)blockIdx.y * a.D + c] = h;
}

template <typename E>
__global__ __launch_bounds__(64) void kda_recurrence_backward_kernel(RecurrenceArgs a) {
    __shared__ float before[kTile][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (c >= a.D) return;
    const Span sp = span_of(a);
    const float* keep = reinterpret_cast<const float*>(a.ws);
    float carry = a.d_state ? a.d_state[(int64_t)blockIdx.y * a.D + c] : 0.f;
    for (int64_t end = sp.end; end > sp.first;) {
        const int64_t tile = (end - 1) / kTile;
        const int64_t lo = tile * kTile > sp.first ? tile * kTile : sp.first;
        float h = lo == sp.first ? (a.state_in ? a.state_in[(int64_t)blockIdx.y * a.D + c] : 0.f)
                                 : keep[(sp.row * tiles_of(a.T) + tile) * a.D + c];
        for (int64_t t = lo; t < end; ++t) {
            const int64_t i = (sp.row * a.T + t) * a.D + c;
            before[t - lo][threadIdx.x] = h;
            h = Decay(fmaxf(a.log_alpha[i], a.floor_)).step(h, to_f32(reinterpret_cast<const E*>(a.x)[i]));
        }
        for (int64_t t = end - 1; t >= lo; --t) {
            const int64_t i = (sp.row * a.T + t) * a.D + c;
            const float la = a.log_alpha[i];
            const Decay decay(fmaxf(la, a.floor_));
            const float d = a.d_out ? to_f32(reinterpret_cast<const E*>(a.d_out)[i]) : 0.f;
            const float hb = before[t - lo][threadIdx.x];
            float s = 1.f;
            if (a.g) {
                s = sigmoidf_(to_f32(reinterpret_cast<const E*>(a.g)[i]));
                const float ht = decay.step(hb, to_f32(reinterpret_cast<const E*>(a.x)[i]));
                reinterpret_cast<E*>(a.dg)[i] = from_f32<E>(d * ht * s * (1.f - s));
            }
            const float dh = fmaf(d, s, carry);
            carry = decay.times(dh);
            reinterpret_cast<E*>(a.dx)[i] = from_f32<E>(dh);
            a.dlog_alpha[i] = la > a.floor_ ? carry * hb : 0.f;
        }
        end = lo;
    }
    if (a.d_state_in) a.d_state_in[(int64_t)blockIdx.y * a.D + c] = carry;
}

template <typename E>
__global__ __launch_bounds__(kThreads) void kda_recurrence_step_kernel(RecurrenceStepArgs a) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.n) return;
    const float h = Decay(fmaxf(a.log_alpha[i], a.floor_)).step(a.state[i], to_f32(reinterpret_cast<const E*>(a.x)[i]));
    a.state[i] = h;
    const float s = a.g ? sigmoidf_(to_f32(reinterpret_cast<const E*>(a.g)[i])) : 1.f;
    reinterpret_cast<E*>(a.out)[i] = from_f32<E>(h * s);
}

}  // namespace

size_t recurrence_workspace_bytes(int64_t B, int64_t T, int64_t D, bool backward) {
    return backward ? (size_t)(B * ((T + kTile - 1) / kTile)) * (size_t)D * sizeof(float) : 0;
}

hipError_t launch_recurrence(bool bf16, const RecurrenceArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.D + 63) / 64), (unsigned)(a.cu_seqlens ? a.n_seq : a.B));
    if (bf16) hipLaunchKernelGGL(kda_recurrence_kernel<__bf16>, grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL(kda_recurrence_kernel<float>, grid, dim3(64), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_recurrence_backward(bool bf16, const RecurrenceArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.D + 63) / 64), (unsigned)(a.cu_seqlens ? a.n_seq : a.B));
    if (bf16) hipLaunchKernelGGL(kda_recurrence_backward_kernel<__bf16>, grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL(kda_recurrence_backward_kernel<float>, grid, dim3(64), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_recurrence_step(bool bf16, const RecurrenceStepArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.n + kThreads - 1) / kThreads));
    if (bf16) hipLaunchKernelGGL(kda_recurrence_step_kernel<__bf16>, grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(kda_recurrence_step_kernel<float>, grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
