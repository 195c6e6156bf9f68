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
// Both calls stream: 8 channels a thread (one 16-byte load of bf16), four
// threads a scale, whose maximum is two lane exchanges.  Bound by HBM.
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

// Row index of a slot within the cache's [pages, heads, page_size] rows, or
// -1 outside it.
__device__ __forceinline__ int64_t row_of(const Cache4Args& c, int64_t slot, int h) {
    if (slot < 0) return -1;
    const int64_t page = slot >> c.page_shift;
    if (page >= c.pages) return -1;
    return ((page * c.heads + h) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
}

// The code (sign and three bits) of y = x / 2^e.
__device__ __forceinline__ uint32_t code_of(float y) {
    const float a = fabsf(y);
    const uint32_t m = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
    return m | ((__float_as_uint(y) >> 31) << 3);
}

template <typename E, int D>
__global__ __launch_bounds__(kThreads) void kda_cache4_append_kernel(Cache4RowsArgs a) {
    constexpr int TPR = D / 8;                 // threads per row
    const int64_t per = a.tokens * a.c.heads * TPR;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= per) return;                      // whole groups of four leave together: per is a multiple of 8
    const int j = (int)(i % TPR);
    const int64_t th = i / TPR;
    const bool v = blockIdx.y == 1;
    const int64_t row = row_of(a.c, a.slot_map[th / a.c.heads], (int)(th % a.c.heads));
    float x[8];
    load8(reinterpret_cast<const E*>(v ? a.v_in : a.k_in) + th * D + 8 * j, x);
    uint32_t m = 0;                            // magnitudes order like their bits; NaN above all
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const bool finite = m < 0x7f800000u;
    int e = (int)(m >> 23) - 127 - 2 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, kScaleLow), kScaleHigh);
    const float unit = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) w |= code_of(x[k] * unit) << (4 * k);
    if (row < 0) return;
    reinterpret_cast<uint32_t*>(v ? a.c.v : a.c.k)[row * TPR + j] = finite ? w : 0u;
    if ((j & 3) == 0) (v ? a.c.v_scale : a.c.k_scale)[row * (D / 32) + j / 4] = finite ? (uint8_t)(e + 127) : 255;
}

template <typename E, int D>
__global__ __launch_bounds__(kThreads) void kda_cache4_read_kernel(Cache4RowsArgs a) {
    constexpr int TPR = D / 8;
    const int64_t per = a.tokens * a.c.heads * TPR;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= per) return;
    const int j = (int)(i % TPR);
    const int64_t th = i / TPR;
    const bool v = blockIdx.y == 1;
    const int64_t row = row_of(a.c, a.slot_map[th / a.c.heads], (int)(th % a.c.heads));
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row >= 0) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(v ? a.c.v : a.c.k)[row * TPR + j];
        const uint32_t b = (v ? a.c.v_scale : a.c.k_scale)[row * (D / 32) + j / 4];
        // 255: NaN; 0: 2^-127, a subnormal
        const float unit = __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t c = w >> (4 * k), m = c & 7u;
            // 0, 1/2, then (1 + bit / 2) 2^(x - 1): exponent x and one mantissa bit
            const float mag = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
            x[k] = (c & 8u ? -mag : mag) * unit;
        }
    }
    store8(reinterpret_cast<E*>(v ? a.v_out : a.k_out) + th * D + 8 * j, x);
}

// Threads of one of K and V: 16 a row of d = 128.
dim3 rows_grid(int d, const Cache4RowsArgs& a) {
    const int64_t threads = a.tokens * a.c.heads * (d / 8);
    return dim3((unsigned)((threads + kThreads - 1) / kThreads), 2);
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
