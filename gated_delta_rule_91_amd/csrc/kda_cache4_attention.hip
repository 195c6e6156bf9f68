// kda_cache4_attention.hip -- causal grouped-query attention over the paged
// 4-bit cache, one wave per (query, head).
//
//   out = sum_t e^(s_t - m) V_t / sum_t e^(s_t - m),  s_t = scale q . K_t,
//   m = max s_t, kept as a running maximum and sum in fp32.
#include "kda_common.hpp"
#include "kda_hybrid_internal.hpp"

namespace kda {

namespace {

__device__ __forceinline__ float value_of(uint32_t code, uint32_t scale) {
    const uint32_t m = code & 7u;
    const float unit = __uint_as_float(scale == 255 ? 0x7fc00000u : scale == 0 ? 0x00400000u : scale << 23);
    const float mag = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    return (code & 8u ? -mag : mag) * unit;
}

// Row index along q that sequence s's queries begin and end at.
__device__ __forceinline__ void rows_of(const Cache4AttentionArgs& a, int64_t s, int64_t& b, int64_t& e) {
    if (!a.cu_seqlens) { b = s; e = s + 1; return; }
    seq_bounds(a.cu_seqlens, s, a.tokens, b, e);
}

template <typename E, int D>
__global__ __launch_bounds__(64) void kda_cache4_attention_kernel(Cache4AttentionArgs a) {
    constexpr int PER = D / 64;
    const int lane = threadIdx.x, head = blockIdx.y, kvh = head / a.group;
    const int64_t row = blockIdx.x;
    int64_t s = 0, b, e;
    if (a.cu_seqlens) {
        int64_t lo = 0, hi = a.n_seq;          // the last sequence that begins at or before the row
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.cu_seqlens[mid] <= row) lo = mid; else hi = mid;
        }
        s = lo;
    } else {
        s = row;
    }
    rows_of(a, s, b, e);
    if (row < b || row >= e) return;
    const int64_t total = a.total_lens[s];
    const int64_t cap = (int64_t)a.max_pages << a.c.page_shift;
    int64_t end = total - (e - b) + (row - b) + 1;      // tokens that the query sees
    end = end < cap ? end : cap;
    float q[PER], o[PER], m = -INFINITY, l = 0.f;
    const int64_t at = (row * a.heads + head) * D;
#pragma unroll
    for (int i = 0; i < PER; ++i) { q[i] = to_f32(reinterpret_cast<const E*>(a.q)[at + lane * PER + i]); o[i] = 0.f; }
    for (int64_t t = 0; t < end; ++t) {
        const int64_t page = a.block_table[s * a.max_pages + (t >> a.c.page_shift)];
        if (page < 0 || page >= a.c.pages) continue;
        const int64_t r = ((page * a.c.heads + kvh) << a.c.page_shift) + (t & ((1 << a.c.page_shift) - 1));
        float dot = 0.f, v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int ch = lane * PER + i;
            const int64_t byte = r * (D / 2) + ch / 2, sc = r * (D / 32) + ch / 32;
            dot += q[i] * value_of(a.c.k[byte] >> (4 * (ch & 1)), a.c.k_scale[sc]);
            v[i] = value_of(a.c.v[byte] >> (4 * (ch & 1)), a.c.v_scale[sc]);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) dot += __shfl_xor(dot, off);
        const float x = dot * a.scale;
        const float mn = x <= m ? m : x;                // a NaN score stays
        const float f = m == -INFINITY ? 0.f : __expf(m - mn), p = mn == -INFINITY ? 0.f : __expf(x - mn);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = o[i] * f + p * v[i];
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        float y = l == 0.f ? 0.f : o[i] / l;
        if (a.g) y *= sigmoidf_(to_f32(reinterpret_cast<const E*>(a.g)[at + lane * PER + i]));
        reinterpret_cast<E*>(a.out)[at + lane * PER + i] = from_f32<E>(y);
    }
}

}  // namespace

size_t cache4_attention_workspace_bytes(int, const Cache4AttentionArgs&) { return 0; }

hipError_t launch_cache4_attention(bool bf16, int d, const Cache4AttentionArgs& a, char*, hipStream_t s) {
    const dim3 grid((unsigned)a.tokens, (unsigned)a.heads);
    if (bf16 && d == 128) hipLaunchKernelGGL((kda_cache4_attention_kernel<__bf16, 128>), grid, dim3(64), 0, s, a);
    else if (bf16) hipLaunchKernelGGL((kda_cache4_attention_kernel<__bf16, 64>), grid, dim3(64), 0, s, a);
    else if (d == 128) hipLaunchKernelGGL((kda_cache4_attention_kernel<float, 128>), grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL((kda_cache4_attention_kernel<float, 64>), grid, dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
