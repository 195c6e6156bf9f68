// kda_plan.hip -- offsets, block tables and slot maps of a serving step, from
// the requests' lengths, in one launch.
//
// With p = page_size, for request r (lengths past_r, new_r):
//   cu_r   = new_0 + ... + new_(r-1)
//   held_r = ceil(past_r / p),  need_r = ceil((past_r + new_r) / p) - held_r
//   first_r = need_0 + ... + need_(r-1)
//   table[r, held_r + j] = free[first_r + j],  j < need_r
//   slot(t) = page * p + pos % p  of token t = cu_r + i, pos = past_r + i,
//             page = table[r, pos / p]
//
// The work is a few KB of lengths and 8 bytes a token: the call is bound by
// latency (256 requests of one token 4.1 us, 512 of up to 509 9.5 us), so it is one launch without a wait between workgroups.  Every
// workgroup forms both prefix sums by itself in LDS (8 bytes a request), and
// a token on a fresh page takes the page off the free list directly instead
// of reading the table entry that another workgroup may be writing.
#include "kda_hybrid_internal.hpp"

namespace kda {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWaves = kPlanThreads / 64;

// The last index i in [0, n) with a[i] <= x, for a[0] = 0 <= x < a[n] and a
// not decreasing.
__device__ __forceinline__ int span_of(const int32_t* a, int n, int64_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kPlanThreads) void kda_plan_kernel(PlanArgs a) {
    extern __shared__ int32_t lds[];
    __shared__ int64_t part[2][kPlanWaves];
    int32_t* cu = lds;                        // [n_req + 1]
    int32_t* first = lds + a.n_req + 1;       // [n_req + 1]
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const bool writer = blockIdx.x == 0;
    const int64_t p1 = ((int64_t)1 << a.page_shift) - 1;

    auto len = [](const int32_t* p, int r) { const int32_t x = p[r]; return (int64_t)(x > 0 ? x : 0); };
    auto pages = [&](int64_t tokens) {
        const int64_t n = (tokens + p1) >> a.page_shift;
        return n < a.max_pages ? n : (int64_t)a.max_pages;
    };

    int64_t sum_new = 0, sum_need = 0;        // over the requests before this stretch
    for (int base = 0; base < a.n_req; base += kPlanThreads) {
        const int r = base + t;
        int64_t n = 0, need = 0;
        if (r < a.n_req) {
            const int64_t past = len(a.past_lens, r);
            n = len(a.new_lens, r);
            need = pages(past + n) - pages(past);
            if (writer) a.total_lens[r] = (int32_t)(past + n < INT32_MAX ? past + n : INT32_MAX);
        }
        int64_t in = n, id = need;            // inclusive sums within the wave
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t un = __shfl_up(in, off), ud = __shfl_up(id, off);
            if (lane >= off) { in += un; id += ud; }
        }
        if (lane == 63) { part[0][wave] = in; part[1][wave] = id; }
        __syncthreads();
        int64_t bn = sum_new, bd = sum_need;
#pragma unroll
        for (int w = 0; w < kPlanWaves; ++w) {
            if (w < wave) { bn += part[0][w]; bd += part[1][w]; }
            sum_new += part[0][w];
            sum_need += part[1][w];
        }
        if (r < a.n_req) {
            const int64_t c = bn + in - n;
            cu[r] = (int32_t)(c < a.tokens ? c : a.tokens);
            first[r] = (int32_t)(bd + id - need);
        }
        __syncthreads();                      // part is read before the next stretch writes it
    }
    if (t == 0) {
        cu[a.n_req] = (int32_t)(sum_new < a.tokens ? sum_new : a.tokens);
        first[a.n_req] = (int32_t)sum_need;
    }
    __syncthreads();
    if (writer) {
        for (int r = t; r <= a.n_req; r += kPlanThreads) a.cu_seqlens[r] = cu[r];
        if (t == 0) a.pages_taken[0] = first[a.n_req];
    }

    const int64_t step = (int64_t)gridDim.x * kPlanThreads, at = (int64_t)blockIdx.x * kPlanThreads + t;
    for (int64_t i = at; i < a.tokens; i += step) {
        int64_t slot = -1;
        if (i < cu[a.n_req]) {
            const int r = span_of(cu, a.n_req, i);
            const int64_t past = len(a.past_lens, r), pos = past + i - cu[r], held = pages(past);
            const int64_t j = pos >> a.page_shift;
            if (j < a.max_pages) {
                int32_t page = -1;
                if (j < held) {
                    page = a.block_table[(int64_t)r * a.max_pages + j];
                } else {
                    const int64_t k = first[r] + j - held;
                    if (k < a.n_free) page = a.free_pages[k];
                }
                if (page >= 0) slot = ((int64_t)page << a.page_shift) + (pos & p1);
            }
        }
        a.slot_map[i] = slot;
    }
    for (int64_t k = at; k < first[a.n_req]; k += step) {
        const int r = span_of(first, a.n_req, k);
        const int64_t j = pages(len(a.past_lens, r)) + k - first[r];
        a.block_table[(int64_t)r * a.max_pages + j] = k < a.n_free ? a.free_pages[k] : -1;
    }
}

}  // namespace

hipError_t launch_plan(const PlanArgs& a, hipStream_t s) {
    // four tokens a thread, up to two workgroups a CU
    const int64_t items = a.tokens > a.n_req ? a.tokens : a.n_req;
    int64_t blocks = (items + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    blocks = blocks < 1 ? 1 : (blocks > 512 ? 512 : blocks);
    const unsigned lds = 2u * (unsigned)(a.n_req + 1) * sizeof(int32_t);
    hipLaunchKernelGGL(kda_plan_kernel, dim3((unsigned)blocks), dim3(kPlanThreads), lds, s, a);
    return hipGetLastError();
}

}  // namespace kda
