// kda_cache4.hip -- rows of keys and values into and out of a paged cache
// held in 4 bits (e2m1 values, a power of two for each 32 channels).
//
//   m = max |x| over 32 channels, e = floor(log2 m) - 2 (+1 where m > 7 * 2^e),
//   kept within [-125, 125];  code = nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 to
//   |x| / 2^e, halves to the even code;  scale byte = e + 127.
// With e = floor(log2 m) - 2 the largest magnitude lies in [4, 8) units: up
// to 7 it is no further from 6 than one unit of the next scale, beyond it the
// next scale is nearer.  Division by 2^e is exact, so a code differs from the
// value by that one rounding only.  The range of e keeps every value
// (1/2 * 2^-125 to 6 * 2^125) a normal number of bf16 and fp32.
//
// Both calls stream: a thread has the same 8 channels of a row's key and value
// (one 16-byte load of bf16 each), four threads a scale, whose maximum is two
// exchanges within the quad.  Bound by HBM: 65536 tokens x 8 heads x 128 in
// bf16 are appended in 85 us (4.0 TB/s) and read in 56 (6.1 TB/s).
#include "kda_common.hpp"
#include "kda_hybrid_internal.hpp"

namespace kda {

namespace {

constexpr int kScaleLow = -125, kScaleHigh = 125;

template <typename E> struct Eight { E x[8]; };

template <typename E>
__device__ __forceinline__ void load8(const E* p, float (&x)[8]) {
    const Eight<E> v = *reinterpret_cast<const Eight<E>*>(__builtin_assume_aligned(p, 16));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(v.x[i]);
}
template <typename E>
__device__ __forceinline__ void store8(E* p, const float (&x)[8]) {
    Eight<E> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x[i] = from_f32<E>(x[i]);
    *reinterpret_cast<Eight<E>*>(__builtin_assume_aligned(p, 16)) = v;
}

// What a thread works on: channels [8 j, 8 j + 8) of row th (token, head), and
// the row of the cache, of its [pages, heads, page_size] rows, or -1.  A
// workgroup has consecutive tokens of one head, whose slots mostly follow each
// other: it writes whole lines of the cache (with tokens and heads the other
// way round the append took 87 us instead of 85, the read 63 instead of 55, on 64K
// tokens x 8 heads; two rows a thread take 89 and 60).
struct Piece {
    int64_t th, row;
    int j;
};
template <int D>
__device__ __forceinline__ bool piece_of(const Cache4RowsArgs& a, Piece& p) {
    constexpr int TPR = D / 8;                 // threads per row
    const int tb = (int)((uint32_t)blockIdx.x / (uint32_t)a.c.heads), h = (int)blockIdx.x - tb * a.c.heads;
    const int64_t token = (int64_t)tb * (kThreads / TPR) + threadIdx.x / TPR;
    p.j = threadIdx.x % TPR;
    if (token >= a.tokens) return false;       // whole rows leave together
    p.th = token * a.c.heads + h;
    const int64_t slot = a.slot_map[token], page = slot >> a.c.page_shift;
    p.row = slot < 0 || page >= a.c.pages ? -1 : ((page * a.c.heads + h) << a.c.page_shift) + (slot & ((1 << a.c.page_shift) - 1));
    return true;
}

// The largest over the lanes of a quad.
__device__ __forceinline__ uint32_t over_quad(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, true));    // lanes 1 0 3 2
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4e, 0xf, 0xf, true)); // lanes 2 3 0 1
}

// The word of 8 codes of x and the scale byte of its quad.
__device__ __forceinline__ void round8(const float (&x)[8], uint32_t& word, uint8_t& scale) {
    uint32_t m = 0;                            // magnitudes order like their bits; NaN above all
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
    m = over_quad(m);
    int e = (int)(m >> 23) - 127 - 2 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, kScaleLow), kScaleHigh);
    // the conversion divides by the scale, rounds halves to the even code and
    // takes magnitudes over 6 as 6
    const float unit = __uint_as_float((uint32_t)(127 + e) << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], unit, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], unit, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], unit, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], unit, 3);
    const bool finite = m < 0x7f800000u;
    word = finite ? w : 0u;
    scale = finite ? (uint8_t)(e + 127) : (uint8_t)255;
}

// What a word of 8 codes stands for, with their scale byte.
__device__ __forceinline__ void values8(uint32_t w, uint32_t scale, float (&x)[8]) {
    const float unit = __uint_as_float(scale << 23);    // only the exponent counts: 0 is 2^-127, 255 NaN
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 3);
    x[0] = a[0]; x[1] = a[1]; x[2] = b[0]; x[3] = b[1]; x[4] = c[0]; x[5] = c[1]; x[6] = d[0]; x[7] = d[1];
}

template <typename E, int D>
__global__ __launch_bounds__(kThreads) void kda_cache4_append_kernel(Cache4RowsArgs a) {
    Piece p;
    if (!piece_of<D>(a, p)) return;
    const int64_t from = p.th * D + 8 * p.j;
    float k[8], v[8];
    load8(reinterpret_cast<const E*>(a.k_in) + from, k);
    load8(reinterpret_cast<const E*>(a.v_in) + from, v);
    uint32_t wk, wv;
    uint8_t sk, sv;
    round8(k, wk, sk);
    round8(v, wv, sv);
    if (p.row < 0) return;
    reinterpret_cast<uint32_t*>(a.c.k)[p.row * (D / 8) + p.j] = wk;
    reinterpret_cast<uint32_t*>(a.c.v)[p.row * (D / 8) + p.j] = wv;
    if ((p.j & 3) == 0) {
        a.c.k_scale[p.row * (D / 32) + p.j / 4] = sk;
        a.c.v_scale[p.row * (D / 32) + p.j / 4] = sv;
    }
}

template <typename E, int D>
__global__ __launch_bounds__(kThreads) void kda_cache4_read_kernel(Cache4RowsArgs a) {
    Piece p;
    if (!piece_of<D>(a, p)) return;
    float k[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (p.row >= 0) {
        const int64_t w = p.row * (D / 8) + p.j, s = p.row * (D / 32) + p.j / 4;
        const uint32_t wk = reinterpret_cast<const uint32_t*>(a.c.k)[w], wv = reinterpret_cast<const uint32_t*>(a.c.v)[w];
        const uint32_t sk = a.c.k_scale[s], sv = a.c.v_scale[s];
        values8(wk, sk, k);
        values8(wv, sv, v);
    }
    const int64_t to = p.th * D + 8 * p.j;
    store8(reinterpret_cast<E*>(a.k_out) + to, k);
    store8(reinterpret_cast<E*>(a.v_out) + to, v);
}

dim3 rows_grid(int d, const Cache4RowsArgs& a) {
    const int per = kThreads / (d / 8);        // rows of a workgroup
    return dim3((unsigned)((a.tokens + per - 1) / per * a.c.heads));
}

}  // namespace

hipError_t launch_cache4_append(bool bf16, int d, const Cache4RowsArgs& a, hipStream_t s) {
    const dim3 grid = rows_grid(d, a);
    if (bf16 && d == 128) hipLaunchKernelGGL((kda_cache4_append_kernel<__bf16, 128>), grid, dim3(kThreads), 0, s, a);
    else if (bf16) hipLaunchKernelGGL((kda_cache4_append_kernel<__bf16, 64>), grid, dim3(kThreads), 0, s, a);
    else if (d == 128) hipLaunchKernelGGL((kda_cache4_append_kernel<float, 128>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((kda_cache4_append_kernel<float, 64>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_cache4_read(bool bf16, int d, const Cache4RowsArgs& a, hipStream_t s) {
    const dim3 grid = rows_grid(d, a);
    if (bf16 && d == 128) hipLaunchKernelGGL((kda_cache4_read_kernel<__bf16, 128>), grid, dim3(kThreads), 0, s, a);
    else if (bf16) hipLaunchKernelGGL((kda_cache4_read_kernel<__bf16, 64>), grid, dim3(kThreads), 0, s, a);
    else if (d == 128) hipLaunchKernelGGL((kda_cache4_read_kernel<float, 128>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((kda_cache4_read_kernel<float, 64>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
