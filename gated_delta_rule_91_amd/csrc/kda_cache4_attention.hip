// kda_cache4_attention.hip -- causal grouped-query attention over the paged
// 4-bit cache, each sequence by itself.  The kernels, what bounds them and what
// they measured are in kda_cache4_attention.hpp.
#include "kda_cache4_attention.hpp"

namespace kda {

namespace {

template <typename E, int D, int R, bool SPLITW>
hipError_t launch_r(const Cache4AttentionArgs& a, const Plan& p, const Parts& parts, hipStream_t s) {
    hipLaunchKernelGGL((kda_cache4_attention_kernel<E, D, R, SPLITW>), dim3((unsigned)(workgroups(p) * a.c.heads)), dim3(kWaves * 64), dynamic_lds(p, D), s, a,
                       p.l, parts);
    return hipGetLastError();
}

template <typename E, int D>
hipError_t launch(const Cache4AttentionArgs& a, char* ws, hipStream_t s) {
    constexpr bool bf16 = sizeof(E) == 2;
    const Plan p = plan_of(bf16, D, a, WHOLE);
    const Parts parts = parts_at(a, p, D, ws);
    hipError_t e;
    if (!p.splitw) e = launch_r<E, D, rows_r(bf16), false>(a, p, parts, s);
    else if (p.r == 1) e = launch_r<E, D, 1, true>(a, p, parts, s);
    else e = launch_r<E, D, 2, true>(a, p, parts, s);
    if (e != hipSuccess || p.l.groups < 2) return e;
    // Where a block has many parts, kWideWaves waves share those of a row:
    // both kernels take 10.7 us instead of 13.3 for one of 4097 tokens (37
    // parts), 16 instead of 18 for 4 of 8192 (16 parts), 28 instead of 112 for
    // one head's 50000; with 4 parts 33 instead of 23 for 8 of 4096, 32 rows.
    const int64_t most = a.group * (a.max_q < a.tokens ? a.max_q : a.tokens);
    const int rows = (int)(most < p.l.rows ? most : p.l.rows);
    const bool wide = p.l.slots * 8 <= p.l.groups;
    const int chunks = wide ? rows : (rows + kWaves - 1) / kWaves;
    const dim3 grid((unsigned)(cuts(p) * a.c.heads * chunks));
    if (wide) hipLaunchKernelGGL((kda_cache4_combine_kernel<E, D, kWideWaves>), grid, dim3(kWideWaves * 64), 0, s, a, p.l, parts, chunks);
    else hipLaunchKernelGGL((kda_cache4_combine_kernel<E, D, 1>), grid, dim3(kWaves * 64), 0, s, a, p.l, parts, chunks);
    return hipGetLastError();
}

}  // namespace

bool cache4_attention_fits(bool bf16, int d, const Cache4AttentionArgs& a) { return attention_fits(bf16, d, a, WHOLE); }

size_t cache4_attention_workspace_bytes(bool bf16, int d, const Cache4AttentionArgs& a) {
    return attention_workspace_bytes(bf16, d, a, WHOLE);
}

hipError_t launch_cache4_attention(bool bf16, int d, const Cache4AttentionArgs& a, char* ws, hipStream_t s) {
    if (bf16) return d == 128 ? launch<__bf16, 128>(a, ws, s) : launch<__bf16, 64>(a, ws, s);
    return d == 128 ? launch<float, 128>(a, ws, s) : launch<float, 64>(a, ws, s);
}

}  // namespace kda
